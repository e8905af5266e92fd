"""Calls of the step metadata and the paged attention at the borders of what include/idx.h allows, on the GPU."""
import threading

import pytest

from test_gpu_attn import Bn, torch  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------ step metadata

def decode_step(torch, Bn, B, T_extra=0, seed=0):
    """The inputs and outputs of a decode step of B requests, its call, and the slots it has to give."""
    P = 64
    g = torch.Generator().manual_seed(seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    ctx = torch.randint(0, 2 * P, (B,), generator=g)
    table = torch.arange(4 * B, **i32).reshape(B, 4).contiguous()
    free = torch.arange(4 * B, 6 * B, **i32)
    T = B + T_extra
    t = dict(ctx=ctx.to(**i32), new=torch.ones(B, **i32), table=table, free=free, span=torch.tensor([0, 2 * B], **i32),
             cu=torch.zeros(B + 1, **i32), lens=torch.zeros(B, **i32), pos=torch.zeros(T, **i32),
             slots=torch.zeros(T, dtype=torch.int64, device="cuda"), nxt=torch.zeros(1, **i32))
    fresh = ctx % P == 0
    order = torch.cumsum(fresh.long(), 0) - 1
    page = torch.where(fresh, 4 * B + order, 4 * torch.arange(B) + ctx // P)
    want = torch.cat([page * P + ctx % P, torch.full((T_extra,), -1)])

    def call(**kw):
        Bn.idx_step_meta(t["ctx"], t["new"], t["table"], P, 4 * P, t["free"], t["span"], 6 * B, t["cu"], t["lens"],
                         t["pos"], t["slots"], t["nxt"], **kw)
    return t, call, want


def test_meta_of_unlike_batches_from_threads(torch, Bn):
    """Host threads whose batches need unlike amounts of shared memory."""
    errors, made = [], [decode_step(torch, Bn, B, 3, B) for B in (16384, 6200, 9000)]
    torch.cuda.synchronize()
    gate = threading.Barrier(len(made))

    def work(t, call, want):
        try:
            stream = torch.cuda.Stream()
            gate.wait()
            for _ in range(1500):
                call(stream=stream)
            stream.synchronize()
            assert torch.equal(t["slots"].cpu(), want)
        except Exception as e:  # seen by the main thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=m) for m in made]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not errors, errors
