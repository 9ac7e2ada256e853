"""The operators at the ends of their ranges: batches without a token at real
widths, losses whose gradient is no number, more logits than one launch forms, both
sides of the rules that choose a kernel, and calls from several host threads."""
import threading

import pytest
import torch

import ops_ref as R
from tensor_adamw_optimizer_amd import _lib as L
from tensor_adamw_optimizer_amd import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def _ffn(t, d, f, dtype, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device=DEV) * std).to(dtype)

    return (normal(t, d), normal(f, d, std=d ** -0.5), normal(f, d, std=d ** -0.5),
            normal(d, f, std=f ** -0.5))


# ---------------------------------------------------------- feed-forward, no tokens

WIDTHS = [(64, 256), (384, 64), (1000, 2731), (1024, 4096), (4096, 1024)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d,f", WIDTHS)
def test_ffn_without_tokens(d, f, dtype):
    """An empty batch (an expert without tokens): no output, zero gradients."""
    x, *w = _ffn(0, d, f, dtype)
    y, kept = ops.gated_ffn_forward(x, *w, keep=True)
    assert y.shape == (0, d)
    for k in (kept, None):
        dx, *dw = ops.gated_ffn_backward(x, x, *w, kept=k)
        assert dx.shape == (0, d)
        for g, t in zip(dw, w):
            assert g.shape == t.shape and not g.any()


@pytest.mark.parametrize("dtype", [L.APEXW_BF16, L.APEXW_F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d,f", WIDTHS)
def test_ffn_without_tokens_through_the_c_abi(d, f, dtype):
    """The same with a place for dx, which has no row to write."""
    _, *w = _ffn(0, d, f, BF if dtype == L.APEXW_BF16 else F32)
    shape = L.apexw_gated_ffn_shape(0, d, f, 0, 0, dtype, L.APEXW_ACT_SILU)
    n = L.apexw_gated_ffn_workspace_bytes(shape, True, False)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
    dw = [torch.full_like(t, 7) for t in w]
    dx = torch.full((d,), 7.0, device=DEV)
    L.apexw_gated_ffn_backward(shape, 0, 0, *(t.data_ptr() for t in w), 0, 0, dx.data_ptr(),
                               *(t.data_ptr() for t in dw), ws.data_ptr(), n,
                               torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert (dx == 7).all() and not any(t.any() for t in dw)


# ---------------------------------------------------------- a loss's gradient that is no number

def _xent(t, d, v, dtype, ignored, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(t, d, generator=gen, device=DEV).to(dtype)
    w = (torch.randn(v, d, generator=gen, device=DEV) * d ** -0.5).to(dtype)
    target = torch.randint(0, v, (t,), generator=gen, device=DEV)
    target[torch.randperm(t, generator=gen, device=DEV)[:int(ignored * t)]] = -100
    return x, w, target


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("t", [5, 70, 2100])
@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_ignored_tokens_under_an_overflowed_loss_scale(reduction, t, dtype, value):
    """A row of dx whose token carries no loss is 0, whatever the loss's gradient;
    so is everything where no token carries one."""
    for ignored in (0.4, 1.0):
        x, w, target = _xent(t, 72, 300, dtype, ignored)
        off = target == -100
        lse = ops.linear_cross_entropy_forward(x, w, target, reduction)[2]
        dloss = torch.full((t,) if reduction == "none" else (), value, device=DEV)
        dx, dw = ops.linear_cross_entropy_backward(x, w, target, lse, dloss, reduction)
        assert off.any() and not dx[off].any() and not dx[off].isnan().any()
        if ignored == 1.0:
            assert not dw.any() and not dw.isnan().any()
        else:
            assert not dx[~off].isfinite().any() and not dw.isfinite().any()


def test_an_ignored_tokens_own_gradient_is_not_looked_at():
    x, w, target = _xent(70, 72, 300, BF, 0.3)
    lse = ops.linear_cross_entropy_forward(x, w, target, "none")[2]
    dloss = torch.rand(70, device=DEV)
    want = ops.linear_cross_entropy_backward(x, w, target, lse, dloss, "none")
    dloss[target == -100] = float("nan")
    got = ops.linear_cross_entropy_backward(x, w, target, lse, dloss, "none")
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---------------------------------------------------------- tokens times vocabulary past one piece

def _scored(x, w, target, sample, got, ignore=-100):
    """Loss and log-sum-exp of the sampled tokens against 64 bits."""
    loss, token, lse = got
    R.within(token[sample], *R.xent(x[sample], w, target[sample], x.dtype, "none", ignore=ignore)[1], "token")
    R.within(lse[sample], *R.xent(x[sample], w, target[sample], x.dtype, "none", ignore=ignore)[2], "lse")
    on = target != ignore
    want = token[on].double().sum() / max(1, int(on.sum()))
    assert abs(loss.double() - want) <= 2 * R.C32 * token[on].double().abs().sum() / max(1, int(on.sum()))
    assert not token[~on].any() and not lse[~on].any()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("t,v", [(16385, 70001), (20000, 131077), (1 << 20, 2500)])
def test_xent_forward_in_pieces_of_the_vocabulary(t, v, dtype):
    """Targets in every piece, at their ends, ignored and outside."""
    x, w, target = _xent(t, 24, v, dtype, 0.2, seed=t)
    got = ops.linear_cross_entropy_forward(x, w, target)
    gen = torch.Generator().manual_seed(3)
    sample = torch.randint(0, t, (300,), generator=gen).to(DEV)
    _scored(x, w, target, sample, got)
    target[sample[:40]] = torch.arange(40, device=DEV) * (v // 40)
    target[sample[40]], target[sample[41]] = v - 1, v
    loss, token, lse = ops.linear_cross_entropy_forward(x, w, target)
    assert loss.isnan() and token[sample[41]].isnan() and int(token.isnan().sum()) == 1
    target[sample[41]] = -100
    _scored(x, w, target, sample, ops.linear_cross_entropy_forward(x, w, target))


def test_xent_forward_of_very_many_tokens_and_classes():
    """More tiles than one launch may have threads for."""
    t, v = 1 << 20, 1 << 19
    x, w, target = _xent(t, 8, v, BF, 0.0, seed=9)
    got = ops.linear_cross_entropy_forward(x, w, target)
    _scored(x, w, target, torch.tensor([0, 1, 77777, t - 2, t - 1], device=DEV), got)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("t", [32, 33, 64, 65])
@pytest.mark.parametrize("d,v", [(2048, 16411), (2050, 16411), (72, 16411)])
def test_xent_on_both_sides_of_a_few_tokens(t, d, v, dtype):
    """Weights large and small, and one whose rows the tiles would have padded."""
    x, w, target = _xent(t, d, v, dtype, 0.2, seed=t)
    target[3] = v - 1
    got = ops.linear_cross_entropy_forward(x, w, target)
    _scored(x, w, target, torch.arange(t, device=DEV), got)


# ---------------------------------------------------------- norm with rotation, grids of few and many tokens

@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("t", [511, 512, 1023, 1024, 1025])
@pytest.mark.parametrize("hq,hk,hd,rotary", [(12, 3, 96, 48), (5, 2, 33, 16)])
def test_qk_on_both_sides_of_many_tokens(t, hq, hk, hd, rotary, dtype):
    gen = torch.Generator(device=DEV).manual_seed(t)
    q, k, dq, dk = (torch.randn(t, h, hd, generator=gen, device=DEV).to(dtype) for h in (hq, hk, hq, hk))
    qw, kw = (torch.rand(hd, generator=gen, device=DEV).to(dtype) + 0.5 for _ in range(2))
    pos = torch.randint(0, 5000, (t,), generator=gen, device=DEV)
    got = [*ops.qk_norm_rope_forward(q, k, qw, kw, pos, rotary_dim=rotary),
           *ops.qk_norm_rope_backward(dq, dk, q, k, qw, kw, pos, rotary_dim=rotary)]
    a = R.qk(q, qw, pos, dtype, rotary=rotary, dy=dq)
    b = R.qk(k, kw, pos, dtype, rotary=rotary, dy=dk)
    for name, x, (want, bound) in zip(("q", "k", "dq", "dk", "dqw", "dkw"), got,
                                      (a[0], b[0], a[1], b[1], a[2], b[2])):
        R.within(x, want, bound, name)


# ---------------------------------------------------------- host threads

def test_two_host_threads_on_two_streams():
    """Shapes and streams of their own, the same plans and tile choices met from
    both sides: each thread's results are those of one thread alone."""
    def work(seed):
        out = []
        for i in range(12):
            t, d, f = 1 + 37 * i, 64 + 8 * i, 96 + 16 * (i % 5)
            x, *w = _ffn(t, d, f, (BF, F32)[i % 2], seed=seed + i)
            y, kept = ops.gated_ffn_forward(x, *w, keep=True)
            out += [y, *ops.gated_ffn_backward(x, x, *w, kept=kept)]
            x, w, target = _xent(t, d, 100 + 301 * i, (BF, F32)[i % 2], 0.2, seed=seed + i)
            a = ops.linear_cross_entropy_forward(x, w, target)
            out += [*a, *ops.linear_cross_entropy_backward(x, w, target, a[2], a[0])]
        return out

    alone = [work(0), work(100)]
    got, wrong = [None, None], []

    def run(n):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(3):
                    got[n] = work(100 * n)
            stream.synchronize()
        except Exception as e:                              # noqa: BLE001
            wrong.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=run, args=(n,)) for n in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong, wrong
    for a, b in zip(alone, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


# ---------------------------------------------------------- graphs

def test_a_released_graph_leaves_no_memory_behind():
    """Shapes first seen under capture, too: what is kept of a call's plan is not in
    the graph's memory, which would then stay for as long as the plan does."""
    def calls(t):
        x, *w = _ffn(t, 64, 96, BF)
        y, kept = ops.gated_ffn_forward(x, *w, keep=True)
        ops.gated_ffn_backward(x, x, *w, kept=kept)
        x, w, target = _xent(t, 64, 300, BF, 0.0)
        lse = ops.linear_cross_entropy_forward(x, w, target)[2]
        ops.linear_cross_entropy_backward(x, w, target, lse, torch.ones((), device=DEV))
        q, pos = x.view(t, 2, 32), target
        ops.qk_norm_rope_backward(q, q, q, q, w[0, :32], w[0, :32], pos)

    def captured(t):
        x, *w = _ffn(t, 64, 96, BF)
        xe, we, target = _xent(t, 64, 300, BF, 0.0)
        one = torch.ones((), device=DEV)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y, kept = ops.gated_ffn_forward(x, *w, keep=True)
            g = ops.gated_ffn_backward(x, x, *w, kept=kept)
            lse = ops.linear_cross_entropy_forward(xe, we, target)[2]
            h = ops.linear_cross_entropy_backward(xe, we, target, lse, one)
            r = ops.qk_norm_rope_backward(*[xe.view(t, 2, 32)] * 4, we[0, :32], we[0, :32], target)
        graph.replay()
        torch.cuda.synchronize()
        del y, kept, g, lse, h, r
        graph.reset()

    def held():
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        return torch.cuda.memory_reserved()

    calls(7)
    captured(7)
    before = held()
    for t in (70, 71, 72):
        captured(t)
    assert held() == before
