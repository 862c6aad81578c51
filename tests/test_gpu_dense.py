"""The dense operators on the GPU against their definition in 64 bits, at the
sizes and inputs where they can go wrong."""
import pytest
import torch

import dense_ref as ref
from gpu_util import DEV, DevLayer, layer_inputs, oracle_forward
from quantized_routed_expert_amd import moe

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
GUARD = 7  # rows around an output that must stay as they were


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def rnd(g, *shape, std=1.0, dtype=BF):
    return ref.scaled(g, *shape, std=std, dtype=dtype, dev=DEV)


class Guarded:
    """A contiguous tensor inside a buffer of sentinels (rows before and behind)."""

    def __init__(self, rows, cols, dtype, like=None, fill=float("nan")):
        self.buf = torch.full((rows + 2 * GUARD, cols), -77.0, dtype=dtype, device=DEV)
        self.t = self.buf[GUARD:GUARD + rows]
        self.t.fill_(fill)
        if like is not None:
            self.t.copy_(like)

    def check(self):
        assert (self.buf[:GUARD] == -77.0).all() and (self.buf[-GUARD:] == -77.0).all(), "rows outside were written"


def nan_around(t):
    """t's values between rows of NaN."""
    buf = torch.full((t.shape[0] + 2 * GUARD, t.shape[1]), float("nan"), dtype=t.dtype, device=t.device)
    buf[GUARD:GUARD + t.shape[0]] = t
    return buf[GUARD:GUARD + t.shape[0]]


SIZES = [(1, 8, 8), (2, 64, 72), (3, 2048, 256), (15, 136, 264), (16, 512, 520), (17, 72, 8), (33, 1000, 520),
         (64, 320, 1032), (65, 264, 128), (127, 128, 136), (128, 8, 1024), (129, 1032, 120), (257, 200, 328),
         (500, 2056, 264)]
BIG = [(1900, 200, 6408), (2100, 264, 5896)]


def linear_case(T, K, N, act, xd, yd, rd, bias, save, seed=0):
    g = gen(seed + T + 3 * K + 7 * N)
    x = nan_around(rnd(g, T, K, dtype=xd))
    w = nan_around(rnd(g, N, K, std=ref.weight_std(K)))
    b = rnd(g, N, std=0.3) if bias else None
    r = nan_around(rnd(g, T, N, dtype=rd)) if rd is not None else None
    ws = moe.linear_workspace(T, K, N)
    y = Guarded(T, N, yd)
    z = Guarded(T, N, BF) if save else None
    moe.linear(x, w, ws, bias=b, act=act, residual=r, z=z.t if save else None, y=y.t)
    torch.cuda.synchronize()
    want = ref.linear(x, w, b, act, r, yd, save)
    ref.check("y", y.t, want["y"])
    y.check()
    if save:
        ref.check("z", z.t, want["z"])
        z.check()


@pytest.mark.parametrize("T,K,N", SIZES + BIG)
def test_linear_sizes(T, K, N):
    i = T % 4
    linear_case(T, K, N, T % 5, BF, (BF, F32)[i & 1], (None, BF, F32, None)[i], i != 2, i >= 2)


@pytest.mark.parametrize("act", range(5))
@pytest.mark.parametrize("T", [4, 150])
def test_linear_acts(T, act):
    linear_case(T, 264, 136, act, BF, BF, F32, True, True)
    linear_case(T, 264, 136, act, F32, F32, BF, True, False)


@pytest.mark.parametrize("T,K,N", [(1, 8, 8), (5, 2048, 256), (16, 72, 136), (37, 1000, 520), (200, 328, 264), (2000, 72, 6408)])
def test_linear_fp32_x(T, K, N):
    linear_case(T, K, N, moe.ACT_NONE, F32, F32, None, False, False)
    linear_case(T, K, N, moe.ACT_SILU, F32, BF, F32, True, True)


def test_linear_fp32_extremes():
    """Each fp32 activation enters whole: the largest and smallest normal values, infinities and NaN in a row of their own."""
    K, N = 64, 8
    x = torch.zeros(8, K, device=DEV)
    x[0, 0], x[1, 1], x[2, 2] = torch.finfo(F32).max, 1.0 + 2.0 ** -23, 1.0 - 2.0 ** -24
    x[3, 3], x[4, 4], x[5, 5], x[6, 6] = 2.0 ** -100 * (2 - 2.0 ** -23), float("inf"), -float("inf"), float("nan")
    w = torch.zeros(N, K, dtype=BF, device=DEV)
    w[:, :8] = 1.0
    y = moe.linear(x, w, moe.linear_workspace(8, K, N))
    torch.cuda.synchronize()
    want = x[:, :8].sum(1, keepdim=True).expand(8, N)
    assert torch.equal(y[:6], want[:6]) and y[6].isnan().all() and (y[7] == 0).all()


def linear_backward_case(T, K, N, act, wd, accumulate, want=("dx", "dw", "dbias")):
    g = gen(T + 5 * K + N)
    x, w = nan_around(rnd(g, T, K)), nan_around(rnd(g, N, K, std=ref.weight_std(K)))
    dy, z = nan_around(rnd(g, T, N, std=0.1)), (nan_around(rnd(g, T, N, std=1.5)) if act else None)
    ws = moe.linear_workspace(T, K, N)
    start = {"dw": rnd(g, N, K, dtype=wd), "dbias": rnd(g, 1, N, dtype=wd)}
    out = {"dx": Guarded(T, K, BF), "dw": Guarded(N, K, wd, start["dw"]), "dbias": Guarded(1, N, wd, start["dbias"])}
    give = {k: (out[k].t[0] if k == "dbias" else out[k].t) for k in want}
    moe.linear_backward(dy, x if "dw" in want else None, w if "dx" in want else None, ws, z=z, act=act, accumulate=accumulate,
                        **give)
    torch.cuda.synchronize()
    r = ref.linear_backward(dy, x, w, z, act, wd)
    for k in want:
        v, e = r[k]
        got = give[k]
        if accumulate and k != "dx":
            s = start[k].reshape(got.shape).double()
            v, e = ref.rounded(v + s, e + 2.0 ** -23 * ((v + s).abs() + e), wd)
        ref.check(k, got, (v, e))
        out[k].check()


@pytest.mark.parametrize("T,K,N", SIZES + [(2000, 520, 264), (100, 4096, 4104), (4200, 72, 40)])
def test_linear_backward_sizes(T, K, N):
    linear_backward_case(T, K, N, T % 5, (BF, F32)[T & 1], (T >> 1) & 1)


@pytest.mark.parametrize("act", range(5))
def test_linear_backward_acts(act):
    linear_backward_case(77, 136, 264, act, F32, False)


@pytest.mark.parametrize("want", [("dx",), ("dw",), ("dbias",), ("dx", "dbias"), ("dw", "dbias")])
def test_linear_backward_parts(want):
    linear_backward_case(40, 72, 136, moe.ACT_GELU, F32, True, want)
    linear_backward_case(40, 72, 136, moe.ACT_NONE, BF, False, want)


def gated_case(T, H, Fw, act, xd, yd, rd, save):
    g = gen(T + 3 * H + Fw)
    x = nan_around(rnd(g, T, H, dtype=xd))
    gate, up = (nan_around(rnd(g, Fw, H, std=ref.weight_std(H))) for _ in range(2))
    down = nan_around(rnd(g, H, Fw, std=ref.weight_std(Fw)))
    r = nan_around(rnd(g, T, H, dtype=rd)) if rd is not None else None
    ws = moe.gated_ffn_workspace(T, H, Fw)
    y, gu = Guarded(T, H, yd), (Guarded(T, 2 * Fw, BF) if save else None)
    moe.gated_ffn(x, moe.dense_ffn(gate, up, down, act), ws, residual=r, gu=gu.t if save else None, y=y.t)
    torch.cuda.synchronize()
    want = ref.gated_ffn(x, gate, up, down, act, r, yd, save)
    ref.check("y", y.t, want["y"])
    y.check()
    if save:
        ref.check("gu", gu.t, want["gu"])
        gu.check()


@pytest.mark.parametrize("T,H,Fw", SIZES + [(1900, 136, 3208), (2100, 2312, 72)])
def test_gated_sizes(T, H, Fw):
    i = T % 4
    gated_case(T, H, Fw, T % 5, BF, (BF, F32)[i & 1], (None, BF, F32, None)[i], i >= 2)


@pytest.mark.parametrize("act", range(5))
def test_gated_acts(act):
    gated_case(3, 264, 136, act, F32, F32, F32, True)
    gated_case(90, 136, 264, act, BF, BF, BF, True)


@pytest.mark.parametrize("T,H,Fw", [(1, 2048, 768), (4, 256, 512), (40, 72, 1032), (1950, 264, 3208)])
def test_gated_fp32_x(T, H, Fw):
    gated_case(T, H, Fw, moe.ACT_SILU, F32, F32, F32, False)
    gated_case(T, H, Fw, moe.ACT_SILU, F32, BF, None, True)


def gated_backward_case(T, H, Fw, act, wd, accumulate, want=("dx", "dgate", "dup", "ddown")):
    g = gen(T + 3 * H + 11 * Fw)
    x, dy = nan_around(rnd(g, T, H)), nan_around(rnd(g, T, H, std=0.1))
    gate, up = (nan_around(rnd(g, Fw, H, std=ref.weight_std(H))) for _ in range(2))
    down = nan_around(rnd(g, H, Fw, std=ref.weight_std(Fw)))
    gu = nan_around(rnd(g, T, 2 * Fw))
    ws = moe.gated_ffn_workspace(T, H, Fw)
    shapes = {"dgate": (Fw, H), "dup": (Fw, H), "ddown": (H, Fw)}
    start = {k: rnd(g, *s, dtype=wd) for k, s in shapes.items()}
    out = {k: Guarded(*shapes[k], wd, start[k]) for k in shapes}
    out["dx"] = Guarded(T, H, BF)
    moe.gated_ffn_backward(dy, x, gu, moe.dense_ffn(gate, up, down, act), ws, accumulate=accumulate,
                           **{k: out[k].t for k in want})
    torch.cuda.synchronize()
    r = ref.gated_ffn_backward(dy, x, gu, gate, up, down, act, wd)
    for k in want:
        v, e = r[k]
        if accumulate and k != "dx":
            s = start[k].double()
            v, e = ref.rounded(v + s, e + 2.0 ** -23 * ((v + s).abs() + e), wd)
        ref.check(k, out[k].t, (v, e))
        out[k].check()


@pytest.mark.parametrize("T,H,Fw", SIZES + [(2000, 520, 264), (100, 2056, 4104), (2048, 264, 6152)])
def test_gated_backward_sizes(T, H, Fw):
    gated_backward_case(T, H, Fw, T % 5, (BF, F32)[T & 1], (T >> 1) & 1)


@pytest.mark.parametrize("act", range(5))
def test_gated_backward_acts(act):
    gated_backward_case(50, 136, 264, act, F32, False)


@pytest.mark.parametrize("want", [("dx",), ("dgate",), ("dup",), ("ddown",), ("dx", "ddown"), ("dgate", "dup")])
def test_gated_backward_parts(want):
    gated_backward_case(40, 72, 136, moe.ACT_SILU, BF, True, want)


# Sizes that take each tile shape, whole and split, in each form (odd tails in all of them).
@pytest.mark.parametrize("T,K,N", [(257, 200, 5584), (130, 136, 5464), (17, 2400, 8), (257, 72, 5448), (2050, 136, 3640),
                                   (130, 2016, 8), (70, 72, 136), (16, 136, 6000), (5, 520, 4200)])
def test_every_tile_forward(T, K, N):
    linear_case(T, K, N, moe.ACT_GELU_TANH, BF, F32, F32, True, True)
    linear_case(T, K, N, moe.ACT_NONE, BF, BF, F32, False, False)
    gated_case(T, K, N, moe.ACT_SILU, BF, BF, BF, True)


@pytest.mark.parametrize("T,H,Fw", [(130, 200, 4168), (70, 72, 4192), (130, 72, 4104), (777, 72, 4136), (16, 72, 4200)])
def test_every_tile_gated(T, H, Fw):
    gated_case(T, H, Fw, moe.ACT_GELU, BF, F32, F32, False)


@pytest.mark.parametrize("T,K,N", [(777, 2352, 200), (777, 584, 7512), (400, 2416, 8), (17, 8, 1800), (777, 2320, 72),
                                   (17, 8, 2024), (2050, 3640, 72)])
def test_every_tile_dx(T, K, N):
    linear_backward_case(T, K, N, moe.ACT_NONE, BF, False, ("dx",))


@pytest.mark.parametrize("T,K,N", [(257, 264, 6608), (17, 136, 5584), (2050, 8, 8), (17, 264, 6608), (17, 1032, 7208), (2050, 96, 8)])
@pytest.mark.parametrize("wd,accumulate", [(BF, False), (F32, True)])
def test_every_tile_dw(T, K, N, wd, accumulate):
    linear_backward_case(T, K, N, moe.ACT_NONE, wd, accumulate, ("dw",))


@pytest.mark.parametrize("T,H,Fw", [(257, 200, 5584), (130, 72, 5464), (17, 1808, 8), (257, 72, 5448), (2050, 72, 3640)])
def test_every_tile_gated_backward(T, H, Fw):
    gated_backward_case(T, H, Fw, moe.ACT_GELU_TANH, BF, False, ("ddown",))
    gated_backward_case(T, H, Fw, moe.ACT_SILU, F32, True)


def test_gradients_together_in_large_tiles():
    linear_backward_case(2100, 2104, 2104, moe.ACT_SILU, F32, True)


def test_offsets_past_32_bits():
    """Rows whose byte offsets pass 2^32 in x, z and y (bf16, 4.4 GB each): the last rows against the definition."""
    T, K, N = 1 << 20, 2104, 2104
    g = gen(9)
    w = rnd(g, N, K, std=ref.weight_std(K))
    x = torch.zeros(T, K, dtype=BF, device=DEV)
    x[-300:] = rnd(g, 300, K)
    ws = moe.linear_workspace(T, K, N)
    y, z = torch.full((T, N), 5.0, dtype=BF, device=DEV), torch.full((T, N), 5.0, dtype=BF, device=DEV)
    moe.linear(x, w, ws, act=moe.ACT_RELU, z=z, y=y)
    torch.cuda.synchronize()
    want = ref.linear(x[-300:], w, None, moe.ACT_RELU, None, BF, True)
    ref.check("y", y[-300:], want["y"])
    ref.check("z", z[-300:], want["z"])
    assert (y[:-300] == 0).all() and (z[:-300] == 0).all()
    dx, dw = torch.empty_like(x), torch.empty(N, K, device=DEV)
    dy = torch.zeros(T, N, dtype=BF, device=DEV)
    dy[-300:] = rnd(g, 300, N, std=0.1)
    moe.linear_backward(dy, x, w, ws, dx=dx, dw=dw)
    torch.cuda.synchronize()
    r = ref.linear_backward(dy[-300:], x[-300:], w, None, moe.ACT_NONE, F32)
    ref.check("dx", dx[-300:], r["dx"])
    ref.check("dw", dw, (r["dw"][0], r["dw"][1]))
    assert (dx[:-300] == 0).all()


def test_no_rows():
    """T = 0: outputs of no rows; weight gradients zero, or as they were when accumulating."""
    K, N = 72, 136
    x, w, dy = torch.empty(0, K, dtype=BF, device=DEV), torch.ones(N, K, dtype=BF, device=DEV), torch.empty(0, N, dtype=BF, device=DEV)
    ws = moe.linear_workspace(0, K, N)
    assert moe.linear(x, w, ws).shape == (0, N)
    for wd in (BF, F32):
        dw, db = torch.full((N, K), 3.0, dtype=wd, device=DEV), torch.full((N,), 3.0, dtype=wd, device=DEV)
        moe.linear_backward(dy, x, w, ws, dx=torch.empty_like(x), dw=dw, dbias=db, accumulate=True)
        assert (dw == 3.0).all() and (db == 3.0).all()
        moe.linear_backward(dy, x, w, ws, dw=dw, dbias=db)
        assert (dw == 0.0).all() and (db == 0.0).all()
    ffn = moe.dense_ffn(w, w, torch.ones(K, N, dtype=BF, device=DEV))
    ws = moe.gated_ffn_workspace(0, K, N)
    assert moe.gated_ffn(x, ffn, ws).shape == (0, K)
    dw = [torch.full(s, 3.0, dtype=BF, device=DEV) for s in ((N, K), (N, K), (K, N))]
    moe.gated_ffn_backward(x, x, torch.empty(0, 2 * N, dtype=BF, device=DEV), ffn, ws, dgate=dw[0], dup=dw[1], ddown=dw[2])
    assert all((d == 0.0).all() for d in dw)


@pytest.mark.parametrize("T", [3, 70, 300])
def test_nan_stays_in_its_row(T):
    g = gen(T)
    H, Fw = 264, 136
    x = rnd(g, T, H)
    ffn = moe.dense_ffn(rnd(g, Fw, H, std=0.06), rnd(g, Fw, H, std=0.06), rnd(g, H, Fw, std=0.1))
    ws = moe.gated_ffn_workspace(T, H, Fw)
    clean = moe.gated_ffn(x, ffn, ws).clone()
    x[T // 2, 5] = float("nan")
    y = moe.gated_ffn(x, ffn, ws)
    torch.cuda.synchronize()
    assert y[T // 2].isnan().all()
    keep = torch.arange(T, device=DEV) != T // 2
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("T", [1, 16, 40, 300])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_residual_in_place(T, dtype):
    g = gen(T)
    H, Fw = 512, 264
    x, r = rnd(g, T, H), rnd(g, T, H, dtype=dtype)
    gate, up, down = rnd(g, Fw, H, std=0.05), rnd(g, Fw, H, std=0.05), rnd(g, H, Fw, std=0.06)
    ws = moe.gated_ffn_workspace(T, H, Fw)
    apart = moe.gated_ffn(x, moe.dense_ffn(gate, up, down), ws, residual=r, y=torch.empty_like(r))
    y = r.clone()
    moe.gated_ffn(x, moe.dense_ffn(gate, up, down), ws, residual=y, y=y)
    torch.cuda.synchronize()
    assert torch.equal(apart, y)


@pytest.mark.parametrize("T", [1, 7, 16, 60, 700])
def test_same_bits_every_run(T):
    g = gen(T)
    H, Fw = 2048, 520
    x, dy = rnd(g, T, H), rnd(g, T, H, std=0.1)
    ffn = moe.dense_ffn(rnd(g, Fw, H, std=0.02), rnd(g, Fw, H, std=0.02), rnd(g, H, Fw, std=0.04))
    ws = moe.gated_ffn_workspace(T, H, Fw)

    def run():
        gu = torch.empty(T, 2 * Fw, dtype=BF, device=DEV)
        out = [moe.gated_ffn(x, ffn, ws, gu=gu), gu, torch.empty_like(x)] + [torch.empty_like(t) for t in ffn.tensors]
        moe.gated_ffn_backward(dy, x, gu, ffn, ws, dx=out[2], dgate=out[3], dup=out[4], ddown=out[5])
        return out

    first = run()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, run()))


def test_workspace_shared_by_sizes_and_operators():
    """One workspace, sized for the largest rows, in turn for other sizes, operators and the routed layer."""
    g = gen(5)
    ly = DevLayer(layer_inputs("tiny", 4))
    H, Fw = 256, 512
    gate, up, down = rnd(g, Fw, H, std=0.06), rnd(g, Fw, H, std=0.06), rnd(g, H, Fw, std=0.05)
    ffn = moe.dense_ffn(gate, up, down)
    n = max(moe.gated_ffn_workspace_bytes(300, H, Fw), moe.linear_workspace_bytes(300, H, Fw),
            moe.workspace_bytes(4, 8, 2, 256, 512, 512))
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    layer = ly.forward()[0]
    for T in (300, 1, 16, 17, 130, 3):
        x = rnd(g, T, H)
        y = moe.gated_ffn(x, ffn, ws)
        ref.check("gated", y, ref.gated_ffn(x, gate, up, down, moe.ACT_SILU, None, BF)["y"])
        v = moe.linear(x, gate, ws)
        ref.check("linear", v, ref.linear(x, gate, None, moe.ACT_NONE, None, BF)["y"])
        assert (ly.forward(ws=ws)[0] == layer).all()


def test_other_stream():
    g = gen(8)
    T, H, Fw = 33, 512, 264
    x = rnd(g, T, H)
    gate, up, down = rnd(g, Fw, H, std=0.05), rnd(g, Fw, H, std=0.05), rnd(g, H, Fw, std=0.06)
    ffn = moe.dense_ffn(gate, up, down)
    ws = moe.gated_ffn_workspace(T, H, Fw)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    a = moe.gated_ffn(x, ffn, ws, stream=side)
    b = moe.linear(x, gate, ws, stream=side.cuda_stream)
    side.synchronize()
    ref.check("gated", a, ref.gated_ffn(x, gate, up, down, moe.ACT_SILU, None, BF)["y"])
    ref.check("linear", b, ref.linear(x, gate, None, moe.ACT_NONE, None, BF)["y"])


def test_null_stream_by_number():
    g = gen(8)
    x, w = rnd(g, 20, 136), rnd(g, 72, 136)
    ws = moe.linear_workspace(20, 136, 72)
    torch.cuda.synchronize()
    y = moe.linear(x, w, ws, stream=0)
    torch.cuda.synchronize()
    ref.check("y", y, ref.linear(x, w, None, moe.ACT_NONE, None, BF)["y"])


def test_block_on_another_device_refused():
    g = gen(2)
    w = rnd(g, 72, 64).cpu()
    x = rnd(g, 4, 64)
    with pytest.raises(ValueError):
        moe.gated_ffn(x, moe.dense_ffn(w, w, w.T.contiguous()), moe.gated_ffn_workspace(4, 64, 72))


@pytest.mark.parametrize("T", [9, 16, 17, 31, 33, 48, 49, 64, 100, 200, 255, 256, 257])
@pytest.mark.parametrize("N", [40, 2048, 5000])
def test_few_rows(T, N):
    """Every share of a window's rows among workgroups."""
    linear_case(T, 264, N, moe.ACT_SILU, BF, BF, F32, True, True)
    linear_case(T, 136, N, moe.ACT_NONE, F32, F32, None, False, False)


def test_binding_refusals():
    g = gen(1)
    x, w, ws = rnd(g, 4, 64), rnd(g, 72, 64), moe.linear_workspace(4, 64, 72)
    for bad in (dict(x=x.T.contiguous().T), dict(w=w.float()), dict(w=w[:, :56]), dict(bias=rnd(g, 64)), dict(residual=rnd(g, 4, 64)),
                dict(residual=rnd(g, 4, 72).half()), dict(z=torch.empty(4, 72, device=DEV)), dict(y=torch.empty(3, 72, dtype=BF, device=DEV)),
                dict(bias=torch.zeros(72, dtype=BF)), dict(ws=ws.float())):
        with pytest.raises((TypeError, ValueError)):
            moe.linear(**{**dict(x=x, w=w, ws=ws), **bad})
    with pytest.raises(moe.MoeError) as e:
        moe.linear(x, w, ws[:4096])
    assert e.value.status == moe.MOE_ERR_WORKSPACE
    with pytest.raises(moe.MoeError):
        moe.linear(x, w, ws, act=9)
    with pytest.raises(TypeError):  # z is needed
        moe.linear_backward(rnd(g, 4, 72), x, w, ws, act=moe.ACT_SILU, dx=torch.empty_like(x))
    with pytest.raises(TypeError):  # one type
        moe.linear_backward(rnd(g, 4, 72), x, w, ws, dw=torch.empty_like(w), dbias=torch.empty(72, device=DEV))
    with pytest.raises(moe.MoeError):  # nothing asked for
        moe.linear_backward(rnd(g, 4, 72), x, w, ws)


def exact_block(T, H, Fw, act):
    """Small whole numbers whose gate and up are exact in bf16, so that the kept values are the definition's own."""
    g = gen(T + H)
    pick = lambda *s: torch.randint(-1, 2, s, generator=g, device=DEV).to(BF)  # noqa: E731
    x, dy = pick(T, H), pick(T, H)
    gate, up, down = pick(Fw, H) * 0.125, pick(Fw, H) * 0.125, pick(H, Fw) * 0.25
    return x, dy, gate, up, down


@pytest.mark.parametrize("act", [moe.ACT_SILU, moe.ACT_GELU, moe.ACT_GELU_TANH])
def test_gated_gradients_against_differences(act):
    """<gradient, direction> against the central difference of <y, dy> in 64 bits.  The difference is off by step^2 / 6 of
    a third derivative (taken at two steps: its own change bounds it), the kernels by their bounds."""
    T, H, Fw = 9, 40, 24
    x, dy, gate, up, down = exact_block(T, H, Fw, act)
    gu = torch.empty(T, 2 * Fw, dtype=BF, device=DEV)
    ws = moe.gated_ffn_workspace(T, H, Fw)
    ffn = moe.dense_ffn(gate, up, down, act)
    moe.gated_ffn(x, ffn, ws, gu=gu)
    out = {"dx": torch.empty_like(x)} | {k: torch.empty_like(t, dtype=F32) for k, t in (("dgate", gate), ("dup", up), ("ddown", down))}
    moe.gated_ffn_backward(dy, x, gu, ffn, ws, **out)
    torch.cuda.synchronize()
    at = {"dx": x.double(), "dgate": gate.double(), "dup": up.double(), "ddown": down.double()}
    assert torch.equal(gu.double(), torch.cat([at["dx"] @ at["dgate"].T, at["dx"] @ at["dup"].T], 1))
    bounds = ref.gated_ffn_backward(dy, x, gu, gate, up, down, act, F32)

    def loss(p):
        h = ref.ACTS[act](p["dx"] @ p["dgate"].T) * (p["dx"] @ p["dup"].T)
        return float((h @ p["ddown"].T * dy.double()).sum())

    for k, got in out.items():
        d = torch.randn(at[k].shape, dtype=torch.float64, generator=gen(3), device=DEV)
        diff = [(loss({**at, k: at[k] + s * d}) - loss({**at, k: at[k] - s * d})) / (2 * s) for s in (1e-4, 2e-4)]
        off = abs(float((got.double() * d).sum()) - diff[0])
        assert off <= float((bounds[k][1] * d.abs()).sum()) + abs(diff[1] - diff[0]) + 1e-6 * abs(diff[0]), k


@pytest.mark.parametrize("act", [moe.ACT_NONE, moe.ACT_SILU, moe.ACT_GELU, moe.ACT_GELU_TANH])
def test_linear_gradients_against_differences(act):
    T, K, N = 9, 40, 24
    x, _, w, _, _ = exact_block(T, K, N, act)
    g = gen(4)
    dy, bias = rnd(g, T, N), (torch.randint(-4, 5, (N,), generator=g, device=DEV) * 0.125).to(BF)
    ws = moe.linear_workspace(T, K, N)
    z = torch.empty(T, N, dtype=BF, device=DEV)
    moe.linear(x, w, ws, bias=bias, act=act, z=z)
    out = {"dx": torch.empty_like(x), "dw": torch.empty_like(w, dtype=F32), "dbias": torch.empty(N, device=DEV)}
    moe.linear_backward(dy, x, w, ws, z=z, act=act, **out)
    torch.cuda.synchronize()
    at = {"dx": x.double(), "dw": w.double(), "dbias": bias.double()}
    assert torch.equal(z.double(), at["dx"] @ at["dw"].T + at["dbias"])
    bounds = ref.linear_backward(dy, x, w, z, act, F32)

    def loss(p):
        return float((ref.ACTS[act](p["dx"] @ p["dw"].T + p["dbias"]) * dy.double()).sum())

    for k, got in out.items():
        d = torch.randn(at[k].shape, dtype=torch.float64, generator=gen(3), device=DEV)
        diff = [(loss({**at, k: at[k] + s * d}) - loss({**at, k: at[k] - s * d})) / (2 * s) for s in (1e-4, 2e-4)]
        off = abs(float((got.double() * d).sum()) - diff[0])
        assert off <= float((bounds[k][1] * d.abs()).sum()) + abs(diff[1] - diff[0]) + 1e-6 * abs(diff[0]), k


def routed_then_shared(T):
    """The routed layer without a shared expert, its output the residual of a bf16 shared expert."""
    li = layer_inputs("tiny", T)
    ly = DevLayer(li)
    cfg = li.cfg
    g = gen(77)
    H, Fw = cfg.hidden, cfg.shared_ffn
    w = rnd(g, Fw, H, std=0.06), rnd(g, Fw, H, std=0.06), rnd(g, H, Fw, std=0.05)
    ffn = moe.dense_ffn(*w)
    ws = torch.zeros(max(moe.workspace_bytes(T, cfg.n_experts, cfg.top_k, H, cfg.ffn, 0), moe.gated_ffn_workspace_bytes(T, H, Fw)),
                     dtype=torch.uint8, device=DEV)
    y = torch.empty(T, H, device=DEV)

    def run():
        moe.layer_forward(ly.x, ly.logits, cfg.top_k, ly.routed, None, y, ws)
        moe.gated_ffn(ly.x, ffn, ws, residual=y, y=y)

    return li, ly, w, ws, y, run


@pytest.mark.parametrize("T", [1, 4, 40])
def test_routed_layer_with_bf16_shared_expert(orc, T):
    li, ly, w, ws, y, run = routed_then_shared(T)
    run()
    torch.cuda.synchronize()
    assert moe.workspace_error(ws) == 0
    cfg = li.cfg
    routed = orc.layer_forward(li.x, li.x_code, li.logits, cfg.top_k, cfg.fmt, cfg.ffn, li.routed, None)[0]
    v, e = ref.gated_ffn(ly.x, *w, moe.ACT_SILU, None, F32)["y"]
    routed = torch.from_numpy(routed).to(DEV).double()
    tol = 2e-3 * routed.square().mean().sqrt()  # the routed layer's own
    ref.check("y", y, (v + routed, e + tol + 2.0 ** -23 * (v + routed).abs()))


@pytest.mark.parametrize("T", [1, 16, 40, 300])
def test_graph_replays(T):
    """A block's forward and backward pass captured once; every replay, on new inputs, with eager calls on the same
    leaves between, equals the eager result."""
    g = gen(T)
    H, Fw = 520, 264
    x, dy = rnd(g, T, H), rnd(g, T, H, std=0.1)
    w = rnd(g, Fw, H, std=0.05), rnd(g, Fw, H, std=0.05), rnd(g, H, Fw, std=0.06)
    ffn = moe.dense_ffn(*w)
    ws, ws2 = moe.gated_ffn_workspace(T, H, Fw), moe.gated_ffn_workspace(T, H, Fw)
    lw, lw2 = moe.linear_workspace(T, H, H), moe.linear_workspace(T, H, H)
    p, bias = rnd(g, H, H, std=0.05), rnd(g, H)

    def outputs():
        e = lambda *s: torch.empty(*s, dtype=BF, device=DEV)  # noqa: E731
        return dict(y=e(T, H), gu=e(T, 2 * Fw), v=e(T, H), z=e(T, H), dv=e(T, H), dp=e(H, H), db=e(H), dx=e(T, H),
                    dgate=e(Fw, H), dup=e(Fw, H), ddown=e(H, Fw))

    def step(o, ws, lw):
        moe.gated_ffn(x, ffn, ws, residual=x, gu=o["gu"], y=o["y"])
        moe.linear(o["y"], p, lw, bias=bias, act=moe.ACT_GELU, z=o["z"], y=o["v"])
        moe.linear_backward(dy, o["y"], p, lw, z=o["z"], act=moe.ACT_GELU, dx=o["dv"], dw=o["dp"], dbias=o["db"])
        moe.gated_ffn_backward(o["dv"], x, o["gu"], ffn, ws, dx=o["dx"], dgate=o["dgate"], dup=o["dup"], ddown=o["ddown"])

    captured, eager = outputs(), outputs()
    step(captured, ws, lw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(captured, ws, lw)
    for i in range(4):
        x.copy_(rnd(g, T, H))
        dy.copy_(rnd(g, T, H, std=0.1))
        step(eager, ws2, lw2)
        graph.replay()
        if i & 1:
            step(eager, ws2, lw2)
        torch.cuda.synchronize()
        for k in captured:
            assert torch.equal(captured[k], eager[k]), (i, k)
