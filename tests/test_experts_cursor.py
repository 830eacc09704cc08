"""The order of the tiled product's loads (host code, compiled here with g++):
every step of every item once, and behind the last item step 0, so that an
empty buffer is never read at an offset."""
import os
import subprocess

from combine_layout_amd import build

PROGRAM = r"""
#include <cstdio>
#include "afd_plan.h"
int main()
{
    for (int nu = 1; nu <= 5; ++nu)
        for (int step = 1; step <= 3; ++step)
            for (int first = 0; first < 3; ++first)
                for (int end = first + 1; end <= first + 7; ++end) {
                    afd::LoadCursor c{first, 0, true};
                    int at = first, u = 0;
                    for (int i = 0; i < 60; ++i) {      // three loads are ahead at most
                        const bool live = at < end;
                        if (c.live != live || c.u != (live ? u : 0) || (live && c.at != at) || c.at >= end) {
                            std::printf("nu %d step %d first %d end %d load %d: at %d u %d live %d\n", nu, step, first, end, i, c.at, c.u, c.live);
                            return 1;
                        }
                        const bool turn = u + 1 == nu && live;
                        if (++u == nu) u = 0, at += step;
                        if (c.advance(nu, end, step) != turn) return 2;
                    }
                }
    return 0;
}
"""


def test_loads_behind_the_last_item_have_no_offset(tmp_path):
    src, exe = tmp_path / "cursor.cpp", tmp_path / "cursor"
    src.write_text(PROGRAM)
    subprocess.check_call(["g++", "-std=c++17", "-Wall", f"-I{build.CSRC}", f"-I{os.path.join(build.ROOT, 'include')}",
                           str(src), "-o", str(exe)])
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout
