"""Which receives Buffer.worker_experts takes: those of the last enqueued
round, whose rows and ends the arena and the workspace hold (over the recording
backend; a receive that is taken fails later, at its host tensors)."""
import pytest
import torch

import combine_layout_amd as afd
from combine_layout_amd import _native as nat
from tests.test_host_core import Ctx


@pytest.fixture
def round_trip():
    """A Buffer over the recording backend, and a round up to its receives."""
    lib = nat.load_fake()
    ctx = Ctx(lib, nat.Config(2, 2, 8, 2, 256, 4, 16, 0, 0, 0))
    buf = afd.Buffer.__new__(afd.Buffer)
    buf.lib, buf.ctx, buf.alpha, buf.K, buf.E, buf._T = lib, ctx.ctx, 4, 2, 8, [4, 4]

    def receive():
        for s in range(2):
            assert ctx.dispatch(s, 4) == 0
        out = []
        for f in range(2):
            st, rec, _ = ctx.receive(f)
            assert st == 0
            rows = torch.zeros(4, 256).bfloat16()
            out.append(afd.Received(rows, None, None, torch.zeros(4, dtype=torch.int32),
                                    nat.Receipt(rec.receipt.round, rec.receipt.partition, 0), rec.receive_rows, None))
        return out

    def finish(recs):
        for f, r in enumerate(recs):
            assert lib.afd_worker_reply(ctx.ctx, f, 0x9000000, r.receive_rows, r.receipt, None) == 0
        for s in range(2):
            assert ctx.collect(s)[0] == 0

    yield buf, receive, finish, ctx
    buf.ctx = None
    ctx.destroy()
    lib.afd_fake_log_clear()


def taken(buf, f, rec):
    with pytest.raises(ValueError, match="on a GPU"):      # only now its host tensors
        buf.worker_experts(f, rec, None)


def test_receives_of_earlier_rounds_are_refused(round_trip):
    buf, receive, finish, ctx = round_trip
    first = receive()
    for f in range(2):
        taken(buf, f, first[f])
    with pytest.raises(ValueError, match="partition"):
        buf.worker_experts(1, first[0], None)
    finish(first)
    taken(buf, 0, first[0])                 # its rows still stand in the arena
    second = receive()
    for f in range(2):
        with pytest.raises(afd.AfdError) as e:
            buf.worker_experts(f, first[f], None)
        assert e.value.status == nat.AFD_E_ORDER
        taken(buf, f, second[f])
    finish(second)
