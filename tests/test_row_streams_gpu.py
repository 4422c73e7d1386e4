"""Row operators one after another on a stream, with programmatic launch on and off."""
import pytest
import torch

import memory_bound_elementwise_gb300 as ew
from tests.rows_util import TORCH, generator, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def restored():
    yield
    ew.set_programmatic_launch(1)


def chain(s, between=lambda: None):
    """Every operator, each on what the one before has just written; all outputs."""
    out = []

    def step(*tensors):
        out.extend(t for t in tensors if t is not None)
        between()
        return tensors

    x, = step(ew.ew_embed(s["table"], s["tokens"], scale=3.0))
    y, h, rstd = step(*ew.ew_rmsnorm(x, s["weight"], residual=s["residual"]))
    q, scales, _, _ = step(*ew.ew_rmsnorm_quant(y, s["weight"], group=64))
    sums, = step(ew.ew_add(y, h))
    logits = sums.view(s["rows"], -1)
    p = step(*ew.ew_logprob(logits, s["picked"], top=7))
    d, = step(ew.ew_logprob_grad(logits, s["picked"], p[2], p[1], p[0], p[1]))
    loss, lse, dl = step(*ew.ew_distill_step(d, s["ids"], s["teacher"], p[1], scale=0.5))
    dl2, = step(ew.ew_distill_grad(dl, s["ids"], s["teacher"], lse, loss))
    dy = dl2.view(y.shape)
    dx, dweight = step(*ew.ew_rmsnorm_grad(dy, h, s["weight"], rstd, dh=sums))
    dtable, = step(ew.ew_embed_grad(dx, s["tokens"], s["table"].shape[0]))
    step(ew.ew_embed_grad(dx, s["tokens"], s["table"].shape[0], dtable=dtable.clone(), accumulate=True))
    return out


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,per", [(12, 512, 3), (600, 2048, 8), (64, 5000, 16)])
def test_chain_with_programmatic_launch_on_and_off(dtype, rows, cols, per):
    kind, n = TORCH[dtype], rows * per
    s = dict(rows=rows, table=randn((300, cols), 91, kind), weight=randn((cols,), 92), residual=randn((n, cols), 93, kind),
             tokens=torch.randint(-1, 300, (n,), generator=generator(94), device="cuda"),
             picked=torch.randint(0, cols * per, (rows,), generator=generator(95), device="cuda"),
             teacher=randn((rows, 40), 96, kind))
    s["ids"] = (s["picked"][:, None] + torch.arange(40, device="cuda") * 7) % (cols * per)
    ew.set_programmatic_launch(0)
    want = chain(s, torch.cuda.synchronize)
    torch.cuda.synchronize()
    for enabled in (0, 1):
        ew.set_programmatic_launch(enabled)
        assert ew.get_programmatic_launch() == enabled
        for stream in (torch.cuda.current_stream(), torch.cuda.Stream()):
            stream.wait_stream(torch.cuda.current_stream())
            for _ in range(3):
                with torch.cuda.stream(stream):
                    got = chain(s)
                stream.synchronize()
                assert len(got) == len(want)
                assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
