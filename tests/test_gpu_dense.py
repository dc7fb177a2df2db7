"""The gated feed-forward block, the cross entropy over a vocabulary and their gradients on the GPU,
value by value against 64 bits, at the sizes, layouts and values where they can go wrong."""
from __future__ import annotations

import pytest
import torch

import dense_reference as ref
import tensor_core_loop_gb300 as tcl

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tcl.lib()
    yield
    assert tcl.last_device_error() == (0, 0)


def laid_out(v, pitch=None, offset=0):
    """v (bf16) with rows `pitch` apart, `offset` elements behind an aligned address; NaN around it."""
    rows, cols = v.shape
    pitch = pitch or cols
    room = torch.full((offset + max(rows - 1, 0) * pitch + cols + 64,), float("nan"), dtype=BF16, device=DEV)
    view = room.as_strided((rows, cols), (pitch, 1), offset)
    view.copy_(v)
    return view


def normal(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).to(BF16).to(DEV)


def block(seed, tokens, hidden, inner):
    g = torch.Generator().manual_seed(seed)
    return (normal(g, tokens, hidden), normal(g, inner, hidden, scale=hidden ** -0.5),
            normal(g, inner, hidden, scale=hidden ** -0.5), normal(g, hidden, inner, scale=inner ** -0.5),
            normal(g, tokens, hidden))


# ------------------------------------------------------------------------------ the feed-forward block

SIZES = [(1, 1, 1), (1, 64, 128), (1, 8, 8), (2, 72, 56), (16, 256, 384), (17, 130, 70), (32, 512, 1000), (33, 1030, 515),
         (64, 320, 4100), (65, 256, 384), (100, 72, 2600), (65, 4096, 10240), (128, 4100, 10243), (128, 64, 64), (129, 64, 136), (256, 128, 256), (257, 1030, 777), (300, 776, 2056), (513, 65, 129),
         (700, 192, 1000)]


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("tokens,hidden,inner", SIZES)
def test_ffn(tokens, hidden, inner, act):
    x, wg, wu, wd, grad = block(tokens + hidden, tokens, hidden, inner)
    out, kept = tcl.gated_ffn(x, wg, wu, wd, activation=act, keep=True)
    want = ref.gated_ffn(x, wg, wu, wd, act)
    for got, w, what in zip((out, kept.gate, kept.up, kept.hidden), want, ("out", "gate", "up", "hidden")):
        assert got.dtype == BF16
        ref.within(got, w, what)
    assert torch.equal(tcl.gated_ffn(x, wg, wu, wd, activation=act), out)
    got = tcl.gated_ffn_grad(grad, x, wg, wu, wd, kept, activation=act)
    for g, w, what in zip(got, ref.gated_ffn_grad(grad, x, wg, wu, wd, act), ("dx", "dw_gate", "dw_up", "dw_down")):
        assert g.dtype == BF16
        ref.within(g, w, what)


# ------------------------------------------------------------------------------ the cross entropy

def tokens_of(seed, tokens, hidden, vocab, spread=1.5, drop=0.1):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(vocab, hidden, generator=g) * spread * hidden ** -0.5
    y = torch.randint(0, vocab, (tokens,), generator=g)
    x = torch.randn(tokens, hidden, generator=g)
    x += 10 * torch.rand(tokens, 1, generator=g) * w[y] / (w[y] ** 2).sum(1, keepdim=True).clamp_min(1e-3)
    y[torch.rand(tokens, generator=g) < drop] = -100
    grad = torch.rand(tokens, generator=g) / tokens
    return x.to(BF16).to(DEV), w.to(BF16).to(DEV), y.to(DEV), grad.to(DEV)


ENTROPY_SIZES = [(1, 1, 1), (1, 64, 1), (1, 64, 500), (3, 8, 31), (16, 256, 5000), (17, 130, 1001), (33, 72, 129), (64, 1030, 700),
                 (65, 128, 64), (100, 64, 128), (128, 72, 20011), (120, 640, 70001), (129, 64, 200), (256, 320, 4096), (257, 130, 3001), (300, 65, 20011), (1000, 512, 257)]


@pytest.mark.parametrize("ids", [torch.int64, torch.int32])
@pytest.mark.parametrize("tokens,hidden,vocab", ENTROPY_SIZES)
def test_entropy(tokens, hidden, vocab, ids):
    x, w, y, grad = tokens_of(tokens + vocab, tokens, hidden, vocab)
    loss, lse = tcl.cross_entropy(x, w, y.to(ids))
    want = ref.cross_entropy(x, w, y)
    ref.within(loss, want[0], "loss")
    ref.within(lse, want[1], "lse")
    got = tcl.cross_entropy_grad(x, w, y.to(ids), grad)
    want = ref.cross_entropy(x, w, y, grad)
    kept = y >= 0
    ref.within(got[0], want[0], "loss")
    ref.within(got[1][kept], ref.V(want[1].v[kept], want[1].e[kept]), "lse")
    ref.within(got[2], want[2], "dx")
    ref.within(got[3], want[3], "dw")


@pytest.mark.parametrize("tokens,hidden,inner,act,dtype", [(300, 3600, 10001, "silu", BF16), (777, 3590, 5000, "gelu", BF16),
                                                            (600, 4100, 7000, "gelu_tanh", F32)])
def test_ffn_of_long_sums(tokens, hidden, inner, act, dtype):
    """More than 56 k-blocks and more tiles than pairs of SMs: tiles of several rounds, longer rings, ends by fewer
    warps."""
    x, wg, wu, wd, grad = block(30, tokens, hidden, inner)
    out, kept = tcl.gated_ffn(x, wg, wu, wd, activation=act, keep=True)
    for got, w, what in zip((out, kept.gate, kept.up, kept.hidden), ref.gated_ffn(x, wg, wu, wd, act), ("out", "gate", "up", "hidden")):
        ref.within(got, w, what)
    got = tcl.gated_ffn_grad(grad, x, wg, wu, wd, kept, activation=act, out_dtype=dtype)
    for g, w, what in zip(got, ref.gated_ffn_grad(grad, x, wg, wu, wd, act, dtype), ("dx", "dw_gate", "dw_up", "dw_down")):
        ref.within(g, w, what)


@pytest.mark.parametrize("tokens,hidden,vocab", [(500, 1030, 20011), (300, 2048, 40000)])
def test_entropy_of_long_sums(tokens, hidden, vocab):
    test_entropy(tokens, hidden, vocab, torch.int64)


# ------------------------------------------------------------------------------ layouts

@pytest.mark.parametrize("tokens", [5, 70, 130])
@pytest.mark.parametrize("extra,offset", [(0, 1), (1, 0), (3, 5), (8, 8), (64, 0)])
def test_ffn_of_rows_at_any_distance_and_address(tokens, extra, offset):
    hidden, inner = 136, 200
    x, wg, wu, wd, grad = block(7, tokens, hidden, inner)
    out, kept = tcl.gated_ffn(x, wg, wu, wd, keep=True)
    want = tcl.gated_ffn_grad(grad, x, wg, wu, wd, kept)
    for which in range(5):
        ops = [laid_out(t, t.shape[1] + extra, offset) if i == which or which == 4 else t for i, t in enumerate((x, wg, wu, wd))]
        g = laid_out(grad, hidden + extra, offset) if which == 4 else grad
        got, k = tcl.gated_ffn(*ops, keep=True)
        assert torch.equal(got, out) and torch.equal(parts(k), parts(kept))
        for a, b in zip(tcl.gated_ffn_grad(g, *ops, k), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("tokens", [5, 70, 130])
@pytest.mark.parametrize("extra,offset", [(0, 1), (1, 0), (3, 5), (8, 8), (64, 0)])
def test_entropy_of_rows_at_any_distance_and_address(tokens, extra, offset):
    x, w, y, grad = tokens_of(8, tokens, 136, 700)
    want = tcl.cross_entropy_grad(x, w, y, grad)
    loss = tcl.cross_entropy(x, w, y)
    for which in range(3):
        a = laid_out(x, 136 + extra, offset) if which != 1 else x
        b = laid_out(w, 136 + extra, offset) if which != 0 else w
        for got, r in zip(tcl.cross_entropy_grad(a, b, y, grad), want):
            assert torch.equal(got, r)
        for got, r in zip(tcl.cross_entropy(a, b, y), loss):
            assert torch.equal(got, r)


def parts(kept):
    """gate, up and hidden, without what lies between their rows."""
    return torch.stack([kept.gate, kept.up, kept.hidden])


def test_kept_rows_at_another_distance():
    x, wg, wu, wd, grad = block(9, 150, 64, 90)
    _, kept = tcl.gated_ffn(x, wg, wu, wd, keep=True)
    want = tcl.gated_ffn_grad(grad, x, wg, wu, wd, kept)
    for pitch in (96, 104, 200):
        room = torch.full((3, 150, pitch), float("nan"), dtype=BF16, device=DEV)
        room[..., :90] = kept.values[..., :90]
        for a, b in zip(tcl.gated_ffn_grad(grad, x, wg, wu, wd, tcl.GatedFfnKept(room, 90)), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("tokens,hidden,inner", [(3, 64, 72), (200, 130, 257)])
def test_ffn_weights_gradients_in_fp32(tokens, hidden, inner):
    x, wg, wu, wd, grad = block(10, tokens, hidden, inner)
    _, kept = tcl.gated_ffn(x, wg, wu, wd, keep=True)
    got = tcl.gated_ffn_grad(grad, x, wg, wu, wd, kept, out_dtype=F32)
    want = ref.gated_ffn_grad(grad, x, wg, wu, wd, "silu", F32)
    assert [t.dtype for t in got] == [BF16, F32, F32, F32]
    for g, w in zip(got, want):
        ref.within(g, w, "gradient")
    for g, h in zip(got[1:], tcl.gated_ffn_grad(grad, x, wg, wu, wd, kept)[1:]):
        assert torch.equal(g.to(BF16), h)


@pytest.mark.parametrize("tokens,hidden,vocab", [(3, 64, 72), (200, 130, 1025)])
def test_entropy_weights_gradient_in_fp32(tokens, hidden, vocab):
    x, w, y, grad = tokens_of(11, tokens, hidden, vocab)
    got = tcl.cross_entropy_grad(x, w, y, grad, out_dtype=F32)
    assert got[3].dtype == F32
    ref.within(got[3], ref.cross_entropy(x, w, y, grad, F32)[3], "dw")
    assert torch.equal(got[3].to(BF16), tcl.cross_entropy_grad(x, w, y, grad)[3])


class Rows:
    """A result with rows `extra` apart, 7 around it."""

    def __init__(self, rows, cols, extra, dtype=BF16):
        self.pitch, self.cols = cols + extra, cols
        self.room = torch.full((rows * self.pitch + 64,), 7.0, dtype=dtype, device=DEV)
        self.view = self.room[: rows * self.pitch].view(rows, self.pitch)

    def args(self):
        return self.room.data_ptr(), self.pitch

    def check(self, want):
        assert torch.equal(self.view[:, : self.cols], want)
        assert (self.view[:, self.cols:] == 7).all() and (self.room[self.view.numel():] == 7).all()


def c_call(fn, *args):
    """Through the C interface, with a workspace of exactly the size that it asks for, surrounded by a pattern."""
    import ctypes
    size = ctypes.c_size_t(0)
    st = fn(*args, None, size, torch.cuda.current_stream().cuda_stream)
    if st == 13:
        room = torch.full((size.value + 512,), 0x5a, dtype=torch.uint8, device=DEV)
        st = fn(*args, room.data_ptr(), size, torch.cuda.current_stream().cuda_stream)
        assert (room[size.value:] == 0x5a).all()
    assert st == 0


@pytest.mark.parametrize("wtype", [0, 1])
@pytest.mark.parametrize("tokens", [5, 100, 300])
@pytest.mark.parametrize("hidden,inner,extra", [(130, 200, 0), (130, 200, 6), (130, 201, 7), (136, 200, 8), (64, 128, 1), (72, 321, 2)])
def test_results_with_wider_rows(tokens, hidden, inner, extra, wtype):
    """What lies between the rows of results stays as it was."""
    from tensor_core_loop_gb300 import dense
    L = dense._lib()
    dtype = F32 if wtype == 0 else BF16
    x, wg, wu, wd, grad = block(31, tokens, hidden, inner)
    out, kept = tcl.gated_ffn(x, wg, wu, wd, keep=True)
    to = Rows(tokens, hidden, extra)
    pitch = kept.values.shape[2]
    mid = torch.empty_like(kept.values)
    h, part = mid.data_ptr(), 2 * tokens * pitch
    ops = [a for t in (x, wg, wu, wd) for a in (t.data_ptr(), t.shape[1])]
    c_call(L.tcl_gated_ffn, tokens, hidden, inner, *ops, 0, h + part, h + 2 * part, h, pitch, *to.args())
    to.check(out)
    assert torch.equal(mid[..., :inner], kept.values[..., :inner])
    want = tcl.gated_ffn_grad(grad, x, wg, wu, wd, kept, out_dtype=dtype)
    res = [Rows(tokens, hidden, extra), Rows(inner, hidden, extra, dtype), Rows(inner, hidden, extra, dtype), Rows(hidden, inner, extra, dtype)]
    c_call(L.tcl_gated_ffn_grad, tokens, hidden, inner, grad.data_ptr(), hidden, *ops, 0, h + part, h + 2 * part, h, pitch,
           *(a for r in res for a in r.args()), wtype)
    for r, w in zip(res, want):
        r.check(w)
    y = torch.randint(0, inner, (tokens,), device=DEV)
    weight = torch.rand(tokens, device=DEV)
    want = tcl.cross_entropy_grad(x, wg, y, weight, out_dtype=dtype)
    loss, lse = torch.empty(2, tokens, device=DEV)
    res = [Rows(tokens, hidden, extra), Rows(inner, hidden, extra, dtype)]
    c_call(L.tcl_cross_entropy_grad, tokens, hidden, inner, *ops[:4], y.data_ptr(), 8, weight.data_ptr(), loss.data_ptr(), lse.data_ptr(),
           *(a for r in res for a in r.args()), wtype)
    for g, w in zip((loss, lse), want):
        assert torch.equal(g, w)
    for r, w in zip(res, want[2:]):
        r.check(w)


# ------------------------------------------------------------------------------ no tokens, dropped tokens, values

def test_no_tokens():
    x, wg, wu, wd, grad = block(12, 0, 72, 130)
    out, kept = tcl.gated_ffn(x, wg, wu, wd, keep=True)
    assert out.shape == (0, 72) and parts(kept).shape == (3, 0, 130)
    for dtype in (BF16, F32):
        dx, *dw = tcl.gated_ffn_grad(grad, x, wg, wu, wd, kept, out_dtype=dtype)
        assert dx.shape == (0, 72) and not any(t.any() for t in dw)
    y, g = torch.empty(0, dtype=torch.int64, device=DEV), torch.empty(0, device=DEV)
    assert all(t.shape == (0,) for t in tcl.cross_entropy(x, wg, y))
    loss, lse, dx, dw = tcl.cross_entropy_grad(x, wg, y, g)
    assert dx.shape == (0, 72) and dw.shape == wg.shape and not dw.any()


@pytest.mark.parametrize("tokens", [7, 64, 120, 300])
def test_dropped_tokens_may_hold_anything(tokens):
    x, w, y, grad = tokens_of(13, tokens, 72, 1000, drop=0.0)
    y[::3] = torch.tensor([-1, 1000, -2 ** 62, 2 ** 62, -100], device=DEV).repeat(tokens)[: y[::3].numel()]
    x[::3] = torch.tensor([float("nan"), float("inf"), -float("inf"), 1e38], device=DEV).repeat(tokens)[: y[::3].numel(), None].to(BF16)
    grad[::6] = float("nan")
    loss, lse, dx, dw = tcl.cross_entropy_grad(x, w, y, grad)
    want = ref.cross_entropy(x, w, y, grad)
    kept = (y >= 0) & (y < 1000)
    assert not loss[~kept].any() and not dx[~kept].any()
    ref.within(loss, want[0], "loss")
    ref.within(dx, want[2], "dx")
    ref.within(dw, want[3], "dw")
    assert torch.equal(tcl.cross_entropy(x, w, y)[0], loss) or tokens <= 128   # (few tokens: another order of the sums)
    ref.within(tcl.cross_entropy(x, w, y)[0], want[0], "loss")


@pytest.mark.parametrize("tokens", [7, 100])
def test_every_token_dropped(tokens):
    x, w, _, grad = tokens_of(14, tokens, 64, 300)
    y = torch.full((tokens,), -100, device=DEV)
    loss, _, dx, dw = tcl.cross_entropy_grad(x, w, y, grad)
    assert not loss.any() and not dx.any() and not dw.any()


def far_logits(seed, tokens, vocab, level, spread):
    """x and w of which the first product of a row and a column sets the logits' level: rows at
    +-level and 0 in turn, chunks of the vocabulary at different heights."""
    g = torch.Generator().manual_seed(seed)
    x, w = torch.randn(tokens, 64, generator=g), torch.randn(vocab, 64, generator=g) * spread / 8
    x[:, 0] = torch.tensor([level, -level, 0.0, level / 2]).repeat(tokens)[:tokens]
    w[:, 0] = 1.0
    w[vocab // 3: vocab // 2, 0] = 0.25
    y = torch.randint(0, vocab, (tokens,), generator=g)
    return x.to(BF16).to(DEV), w.to(BF16).to(DEV), y.to(DEV), (torch.rand(tokens, generator=g) / tokens).to(DEV)


@pytest.mark.parametrize("tokens", [9, 90, 150])
@pytest.mark.parametrize("level,spread", [(40.0, 1.0), (64.0, 8.0), (90.0, 1.0), (300.0, 20.0), (20000.0, 1.0)])
def test_logits_far_from_zero(tokens, level, spread):
    """Exponentials that leave fp32's range without their largest logit taken out, and chunks of one row that
    do so while others do not."""
    x, w, y, grad = far_logits(15, tokens, 1100, level, spread)
    want = ref.cross_entropy(x, w, y, grad)
    for got in (tcl.cross_entropy(x, w, y), tcl.cross_entropy_grad(x, w, y, grad)):
        for g, r, what in zip(got, want, ("loss", "lse", "dx", "dw")):
            ref.within(g, r, what)


def test_masked_vocabulary():
    """Columns at minus infinity (a masked part of the vocabulary) have no weight."""
    x, w, y, _ = tokens_of(16, 200, 64, 900, drop=0.0)
    x[:, 0], w[:, 0] = 1.0, 0.0
    w[256:700, 0] = -float("inf")
    y = torch.where((y >= 256) & (y < 700), y % 256, y)
    keep = torch.cat([w[:256], w[700:]])
    z = torch.where(y >= 700, y - 444, y)
    for n in (10, 100, 200):
        got = tcl.cross_entropy(x[:n], w, y[:n])
        want = ref.cross_entropy(x[:n], keep, z[:n])
        for g, r in zip(got, want):
            ref.within(g, r, "loss")


def test_nan_stays_in_its_row():
    x, w, y, _ = tokens_of(17, 200, 64, 500, drop=0.0)
    wg, wu = w[:300], w[200:]
    wd = w.t()[:, :300].contiguous()
    out = tcl.gated_ffn(x, wg, wu, wd)
    loss = tcl.cross_entropy(x, w, y)[0]
    x[33] = float("nan")
    rows = torch.arange(200, device=DEV) != 33
    for n in (200, 100, 50):
        got = tcl.gated_ffn(x[:n], wg, wu, wd)
        assert got[33].isnan().all()
        full = torch.equal(got[rows[:n]], out[:n][rows[:n]])
        assert full or n <= 128   # (few tokens: another order of the sums)
        assert got[rows[:n]].isfinite().all()
        got = tcl.cross_entropy(x[:n], w, y[:n])[0]
        assert got[33].isnan() and got[rows[:n]].isfinite().all()
    assert torch.equal(tcl.cross_entropy(x, w, y)[0][rows], loss[rows])


@pytest.mark.parametrize("tokens", [200, 2100])
@pytest.mark.parametrize("target", [0, 7])
def test_infinite_logit_is_not_lost(tokens, target):
    """One token with one logit of infinity (minus infinity for the others): its gradients are no numbers."""
    x, w, y, grad = tokens_of(27, tokens, 64, 500, drop=0.0)
    x[:, 0], w[:, 0] = -1.0, 0.0
    x[33, 0], w[7, 0], y[33] = 1.0, float("inf"), target
    y = torch.where((y == 7) & (torch.arange(tokens, device=DEV) != 33), 8, y)
    loss, lse, dx, dw = tcl.cross_entropy_grad(x, w, y, grad)
    assert float(lse[33]) == float("inf") and not loss[33].isfinite()
    assert dx[33].isnan().all() and dw.isnan().all()
    others = torch.arange(tokens, device=DEV) != 33
    assert loss[others].isfinite().all() and dx[others][:, 1:].isfinite().all()


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activations_over_their_whole_range(act):
    """One hidden value and weights of one: gates of every size, up to where the results end."""
    v = torch.cat([torch.linspace(-20, 20, 4001), torch.tensor([1e-30, -1e-30, 3e3, -3e3, 1e5, -1e5, 1e18, -1e18, 0.0, -0.0])])
    x = torch.zeros(v.numel(), 8, dtype=BF16, device=DEV)
    x[:, 0] = v.to(BF16).to(DEV)
    x[:, 1] = 1.0
    eye = torch.eye(8, dtype=BF16, device=DEV)
    wg, wu, wd = eye[:1].contiguous(), eye[1:2].contiguous(), eye[:, :1].contiguous()
    out, kept = tcl.gated_ffn(x, wg, wu, wd, activation=act, keep=True)
    want = ref.gated_ffn(x, wg, wu, wd, act)
    ref.within(out, want[0], "out")
    grad = torch.zeros_like(x)
    grad[:, 0] = 1.0
    got = tcl.gated_ffn_grad(grad, x, wg, wu, wd, kept, activation=act)
    ref.within(got[0], ref.gated_ffn_grad(grad, x, wg, wu, wd, act)[0], "dx")


# ------------------------------------------------------------------------------ large sizes

def test_many_tokens_over_few_words_take_little_memory():
    """A workspace of some values for each token, at the first call."""
    tokens = 300_000
    x, w, y, _ = tokens_of(29, tokens, 64, 100)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    tcl.cross_entropy(x, w, y)
    assert torch.cuda.max_memory_allocated() - before <= tokens * (8 * 2 + 4 + 4 + 4) + 2 ** 22


def test_exponentials_in_pieces():
    """More than 2 GiB of exponentials: the pieces' gradients of w are added in fp32."""
    tokens, vocab = 8192 + 300, 131072
    x, w, y, grad = tokens_of(18, tokens, 64, vocab)
    loss, lse, dx, dw = tcl.cross_entropy_grad(x, w, y, grad)
    total = torch.zeros(vocab, 64, dtype=torch.float64, device=DEV)
    bound = torch.zeros_like(total)
    for i in range(0, tokens, 2048):
        p = slice(i, i + 2048)
        want = ref.cross_entropy(x[p], w, y[p], grad[p], F32)
        ref.within(loss[p], want[0], "loss")
        ref.within(dx[p], want[2], "dx")
        total += want[3].v
        bound += want[3].e + 2.0 ** -23 * want[3].v.abs()
    ref.within(dw, ref.rounded(ref.V(total, bound)), "dw")


def test_as_many_tokens_as_there_may_be():
    """The last piece's end passes 32 bits. Only some tokens, first, last and at the pieces' ends, have a
    weight."""
    tokens, vocab, piece = 2 ** 31 - 2 ** 16 - 1, 512, 2 ** 21
    g = torch.Generator(device=DEV).manual_seed(28)
    x = torch.zeros(tokens, 8, dtype=BF16, device=DEV)[:, :1]   # (rows of one value on 16-byte pieces)
    w = (torch.randn(vocab, 1, device=DEV, generator=g)).to(BF16)
    y = torch.full((tokens,), -1, dtype=torch.int32, device=DEV)
    grad = torch.zeros(tokens, device=DEV)
    some = torch.cat([torch.arange(i, i + 40, device=DEV) for i in (0, piece - 20, 512 * piece - 20, 1023 * piece - 20, tokens - 40)])
    x[some] = torch.randn(some.numel(), 1, device=DEV, generator=g).to(BF16)
    y[some] = torch.randint(0, vocab, (some.numel(),), device=DEV, generator=g).int()
    grad[some] = torch.rand(some.numel(), device=DEV, generator=g)
    loss, lse, dx, dw = tcl.cross_entropy_grad(x, w, y, grad)
    want = ref.cross_entropy(x[some], w, y[some], grad[some])
    for got, r, what in zip((loss[some], lse[some], dx[some], dw), want, ("loss", "lse", "dx", "dw")):
        ref.within(got, r, what)
    assert int((loss != 0).sum()) <= some.numel() and int((dx != 0).sum()) <= some.numel()


def test_weights_past_32_bits_of_elements():
    tokens, hidden, vocab = 70, 4096, 540_000
    g = torch.Generator(device=DEV).manual_seed(19)
    x = torch.randn(tokens, hidden, device=DEV, generator=g).to(BF16)
    w = torch.empty(vocab, hidden, dtype=BF16, device=DEV)
    for i in range(0, vocab, 60_000):
        w[i:i + 60_000] = torch.randn(60_000, hidden, device=DEV, generator=g) * 0.02
    y = torch.randint(vocab - 2000, vocab, (tokens,), device=DEV, generator=g)
    grad = torch.rand(tokens, device=DEV, generator=g) / tokens
    loss, lse, dx, dw = tcl.cross_entropy_grad(x, w, y, grad)
    l = torch.cat([x.double() @ w[i:i + 60_000].double().t() for i in range(0, vocab, 60_000)], 1)
    want = torch.logsumexp(l, 1)
    error = float(ref.unit(hidden) * (x.double().abs() @ w[:1000].double().abs().t()).max()) * 1.5 + 1e-5
    assert ((lse - want).abs() <= error).all()
    assert ((loss - (want - l.gather(1, y[:, None])[:, 0])).abs() <= 2 * error).all()
    rows = torch.cat([torch.arange(300, device=DEV), torch.arange(vocab - 2000, vocab, device=DEV)])
    d = torch.exp(l[:, rows] - want[:, None])
    d -= (rows == y[:, None]).double()
    d *= grad.double()[:, None]
    far = ref.rounded(ref.matmul(ref.V(d.t(), d.t().abs() * (ref.BF + 2 * error)), ref.V(x.double(), ref.BF * x.double().abs())))
    ref.within(dw[rows], far, "dw")
    few = tcl.cross_entropy(x[:5], w, y[:5])
    assert ((few[1] - want[:5]).abs() <= error).all()


def test_kept_past_32_bits_of_elements():
    tokens, hidden, inner = 262_200, 64, 8320
    g = torch.Generator(device=DEV).manual_seed(20)
    x = torch.randn(tokens, hidden, device=DEV, generator=g).to(BF16)
    wg, wu = ((torch.randn(inner, hidden, device=DEV, generator=g) / 8).to(BF16) for _ in range(2))
    wd = (torch.randn(hidden, inner, device=DEV, generator=g) / 90).to(BF16)
    grad = torch.randn(tokens, hidden, device=DEV, generator=g).to(BF16)
    out, kept = tcl.gated_ffn(x, wg, wu, wd, keep=True)
    dx, dwg, dwu, dwd = tcl.gated_ffn_grad(grad, x, wg, wu, wd, kept, out_dtype=F32)
    for p in (slice(0, 200), slice(tokens - 200, tokens)):
        for a, b in zip((out[p], kept.gate[p], kept.up[p], kept.hidden[p]), ref.gated_ffn(x[p], wg, wu, wd, "silu")):
            ref.within(a, b, "forward")
        ref.within(dx[p], ref.gated_ffn_grad(grad[p], x[p], wg, wu, wd, "silu")[0], "dx")
    # Eight columns of h, summed over all tokens. An fp32 sum errs in each of its additions by 2^-23 of the partial
    # sum at most (of one that starts anywhere, where K is cut into ranges): twice the largest one from the
    # start on, and the 16 products that an MMA adds to it.
    some = slice(inner - 8, inner)
    r = ref.gated_ffn(x, wg[some], wu[some], wd[:, some], "silu")
    gx, xx = ref.exactly(grad), ref.exactly(x)
    dh = ref.matmul(gx, ref.exactly(wd[:, some]))
    a, slope = ref.act("silu", r[1])
    dg, du = ref.rounded(ref.times(ref.times(dh, r[2]), slope)), ref.rounded(ref.times(dh, a))
    for got, left, right in ((dwg[some], dg, xx), (dwu[some], du, xx), (dwd[:, some].t(), r[3], gx)):
        product = left.v[:, :, None] * right.v[:, None, :]
        sums = product.cumsum(0)
        bound = left.e.t() @ right.v.abs() + ref.unit(tokens) * 2 * (sums.abs().amax(0) + 16 * product.abs().amax(0))
        ref.within(got, ref.V(sums[-1], bound), "weights' gradient")


# ------------------------------------------------------------------------------ streams, graphs, threads

def step(x, gate, up, down, table, targets, grad):
    """A training step's dense part: block with a residual, loss, gradients, clipping."""
    out, kept = tcl.gated_ffn(x, gate, up, down, keep=True)
    y = x + out
    loss, lse, dy, dtable = tcl.cross_entropy_grad(y, table, targets, grad)
    dx, *dw = tcl.gated_ffn_grad(dy, x, gate, up, down, kept)
    grads = [*dw, dtable]
    before = [t.clone() for t in grads]
    norm = tcl.clip_grads(grads, 0.01)
    return dict(out=out, kept=kept, y=y, loss=loss, dy=dy, dx=dx, before=before, grads=grads, norm=norm)


def operands(seed, tokens, hidden, inner, vocab):
    x, gate, up, down, _ = block(seed, tokens, hidden, inner)
    _, table, targets, grad = tokens_of(seed, tokens, hidden, vocab)
    return x, gate, up, down, table, targets, grad


def flat(r):
    return [r["out"], parts(r["kept"]), r["loss"], r["dy"], r["dx"], *r["before"], *r["grads"], r["norm"]]


@pytest.mark.parametrize("tokens,hidden,inner,vocab", [(48, 64, 200, 333), (300, 136, 384, 2050)])
def test_training_step(tokens, hidden, inner, vocab):
    """The calls one after another, each against 64 bits of what it was given, eager and captured."""
    ops = operands(21, tokens, hidden, inner, vocab)
    x, gate, up, down, table, targets, grad = ops
    r = step(*ops)
    for a, b in zip((r["out"], *parts(r["kept"])), ref.gated_ffn(x, gate, up, down, "silu")):
        ref.within(a, b, "block")
    loss, _, dy, dtable = ref.cross_entropy(r["y"], table, targets, grad)
    ref.within(r["loss"], loss, "loss")
    ref.within(r["dy"], dy, "dy")
    ref.within(r["before"][3], dtable, "dtable")
    for a, b in zip((r["dx"], *r["before"][:3]), ref.gated_ffn_grad(r["dy"], x, gate, up, down, "silu")):
        ref.within(a, b, "gradient")
    norm = float(sum((t.double() ** 2).sum() for t in r["before"])) ** 0.5
    assert norm > 0.01 and abs(float(r["norm"]) - norm) <= 20 * 2.0 ** -24 * norm
    for t, g in zip(r["before"], r["grads"]):
        exact = t.double() * (0.01 / norm)
        assert ((g.double() - exact).abs() <= (ref.BF + 2.0 ** -19) * exact.abs() + ref.TINY).all()

    # captured, and replayed with other tokens in the same places
    static = [t.clone() for t in ops]
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        held = step(*static)
    for seed in (21, 22):
        fresh = operands(seed, tokens, hidden, inner, vocab)
        for s, t in zip(static, fresh):
            s.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(flat(held), flat(step(*fresh))):
            assert torch.equal(a, b)


def test_same_bits_again():
    ops = operands(23, 513, 320, 1000, 5003)
    first = flat(step(*ops))
    for _ in range(3):
        for a, b in zip(first, flat(step(*ops))):
            assert torch.equal(a, b)


def test_streams_side_by_side():
    """Steps of different sizes on two streams and the current one, without any order between them."""
    jobs = [operands(24, 300, 136, 384, 2050), operands(25, 20, 1030, 515, 700), operands(26, 1000, 256, 1030, 9001)]
    alone = [[t.clone() for t in flat(step(*ops))] for ops in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.current_stream()]
    got = []
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((i, flat(step(*jobs[i]))))
    torch.cuda.synchronize()
    for i, r in got:
        for a, b in zip(r, alone[i]):
            assert torch.equal(a, b)


def test_given_stream():
    """Calls on a stream that is not the current one, whose operands are dropped right after."""
    ops = operands(27, 200, 130, 300, 1500)
    x, gate, up, down, table, targets, grad = ops
    out, kept = tcl.gated_ffn(x, gate, up, down, keep=True)
    want = [out, *tcl.cross_entropy(x, table, targets), *tcl.cross_entropy_grad(x, table, targets, grad),
            *tcl.gated_ffn_grad(x, x, gate, up, down, kept), tcl.grad_norm([gate, up])]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = [t.clone() for t in ops]
    s.wait_stream(torch.cuda.current_stream())
    o, k = tcl.gated_ffn(*a[:4], keep=True, stream=s)
    got = [o, *tcl.cross_entropy(a[0], a[4], a[5], stream=s), *tcl.cross_entropy_grad(a[0], a[4], a[5], a[6], stream=s),
           *tcl.gated_ffn_grad(a[0], *a[:4], k, stream=s), tcl.grad_norm(a[1:3], stream=s)]
    del a, k
    junk = [torch.full_like(t, 3) for t in ops]   # (takes the memory if it was given back)
    s.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)
    del junk


@pytest.mark.parametrize("tokens", [5, 300])
def test_given_stream_and_current_one_give_the_same_bits(tokens):
    """Two ways through the binding."""
    x, wg, wu, wd, grad = block(31, tokens, 72, 200)
    xe, w, y, ge = tokens_of(31, tokens, 72, 500)
    st = torch.cuda.current_stream()
    for dtype in (None, BF16, F32):
        out, kept = tcl.gated_ffn(x, wg, wu, wd, activation="gelu", keep=True)
        again, kept_again = tcl.gated_ffn(x, wg, wu, wd, activation="gelu", keep=True, stream=st)
        pairs = [(out, again), (kept.hidden, kept_again.hidden), (kept.gate, kept_again.gate), (kept.up, kept_again.up)]
        pairs += [(out, tcl.gated_ffn(x, wg, wu, wd, activation="gelu"))]
        args = (grad, x, wg, wu, wd, kept, "gelu", dtype)
        pairs += zip(tcl.gated_ffn_grad(*args), tcl.gated_ffn_grad(*args, stream=st))
        pairs += zip(tcl.cross_entropy(xe, w, y), tcl.cross_entropy(xe, w, y, stream=st))
        pairs += zip(tcl.cross_entropy_grad(xe, w, y, ge, dtype), tcl.cross_entropy_grad(xe, w, y, ge, dtype, stream=st))
        grads = [a.clone() for a, _ in pairs]
        outs = [[torch.empty_like(a) for a in grads] for _ in range(2)]
        pairs += [(tcl.clip_grads(grads, 1, out=outs[0]), tcl.clip_grads(grads, 1, out=outs[1], stream=st)), *zip(*outs)]
        for a, b in pairs:
            assert a.dtype == b.dtype and a.shape == b.shape and torch.equal(a, b)


def test_two_threads():
    import threading
    jobs = [operands(28, 300, 136, 384, 2050), operands(29, 40, 1030, 515, 700)]
    alone = [[t.clone() for t in flat(step(*ops))] for ops in jobs]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(10):
                r = flat(step(*jobs[i]))
                s.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(r, alone[i])):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_same_memory_for_gate_and_up():
    """One matrix as both weights, one tensor as x and grad: nothing says that they may not be."""
    x, wg, _, wd, _ = block(30, 130, 136, 200)
    out, kept = tcl.gated_ffn(x, wg, wg, wd, keep=True)
    ref.within(out, ref.gated_ffn(x, wg, wg, wd, "silu")[0], "out")
    for a, b in zip(tcl.gated_ffn_grad(x, x, wg, wg, wd, kept), ref.gated_ffn_grad(x, x, wg, wg, wd, "silu")):
        ref.within(a, b, "gradient")


FIRST = """
import torch, tensor_core_loop_gb300 as tcl
dev = torch.device("cuda:0")
t = lambda *s: torch.full(s, 0.01, dtype=torch.bfloat16, device=dev)
n = {tokens}
x, wg, wd, table = t(n, 64), t(200, 64), t(64, 200), t(300, 64)
y, grad = torch.zeros(n, dtype=torch.int64, device=dev), torch.ones(n, device=dev)
tcl.lib()
s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(g, stream=s):
    out, kept = tcl.gated_ffn(x, wg, wg, wd, keep=True)
    grads = tcl.gated_ffn_grad(x, x, wg, wg, wd, kept)
    loss = tcl.cross_entropy(out, table, y)
    more = tcl.cross_entropy_grad(out, table, y, grad)
    norm = tcl.clip_grads([*grads, more[3]], 1e-3)
g.replay()
torch.cuda.synchronize()
held = [out, *loss, *more[:3], norm]
out2, kept = tcl.gated_ffn(x, wg, wg, wd, keep=True)
more2 = tcl.cross_entropy_grad(out2, table, y, grad)
norm2 = tcl.clip_grads([*tcl.gated_ffn_grad(x, x, wg, wg, wd, kept), more2[3]], 1e-3)
for a, b in zip(held, [out2, *tcl.cross_entropy(out2, table, y), *more2[:3], norm2]):
    assert torch.equal(a, b)
assert tcl.last_device_error() == (0, 0)
"""


@pytest.mark.parametrize("tokens", [5, 200])
def test_first_calls_of_a_process_inside_a_capture(tokens):
    """Nothing has to be set up by a call before: no scratch, no attribute, no measurement."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST.format(tokens=tokens)], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("tokens", [16, 300])
def test_losses_are_fp32_sums(tokens):
    """The target's logit is an fp32 sum of 16 products to a thread (4096 of them) and five to eight more
    additions: off by 26 roundings of 2^-24 of the products' magnitudes at most. lse is off by the other
    logits' errors, which the softmax averages: here below 2^-21 of it."""
    x, w, y, _ = tokens_of(32, tokens, 4096, 3000, spread=2.0, drop=0.0)
    x[::2] += (12 * w[y[::2]].double() / (w[y[::2]].double() ** 2).sum(1, keepdim=True)).to(BF16)   # (near-certain ones)
    l = x.double() @ w.double().t()
    lse = torch.logsumexp(l, 1)
    want = lse - l.gather(1, y[:, None])[:, 0]
    size = (x.double().abs() * w[y].double().abs()).sum(1)
    for got in (tcl.cross_entropy(x, w, y)[0], tcl.cross_entropy_grad(x, w, y, torch.ones(tokens, device=DEV))[0]):
        assert ((got.double() - want).abs() <= 26 * 2.0 ** -24 * size + 2.0 ** -21 * lse).all()
