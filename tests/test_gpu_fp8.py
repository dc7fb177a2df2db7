"""The e4m3 quantising and products on the GPU against their definitions in 64 bits."""
from __future__ import annotations

import pytest
import torch

import fp8_reference as ref
import tensor_core_loop_gb300 as tcl

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tcl.lib()
    yield
    assert tcl.last_device_error() == (0, 0)


def numbers(rows, cols, seed, dtype=BF16, batch=None):
    g = torch.Generator().manual_seed(seed)
    shape = (rows, cols) if batch is None else (batch, rows, cols)
    x = torch.randn(shape, generator=g) * torch.exp(2 * torch.randn(cols, generator=g))
    return x.to(dtype)


def random_operand(rows, cols, seed, per=1, pitch=None, scale_layout="groups", batch=None):
    """e4m3 data of any bit pattern but NaN, with scales over a few powers of two."""
    g = torch.Generator().manual_seed(seed)
    lead = () if batch is None else (batch,)
    bits = torch.randint(0, 254, lead + (rows, pitch or cols), generator=g, dtype=torch.uint8)
    bits = torch.where(bits >= 127, bits + 1, bits)     # 0x7f and 0xff are NaN
    data = bits.view(F8).to(DEV)[..., :cols]
    sr = -(-rows // per)
    scale = torch.exp2(3 * torch.randn(lead + (sr, ref.groups(cols)), generator=g)).to(DEV)
    if scale_layout == "groups":
        scale = scale.transpose(-1, -2).contiguous().transpose(-1, -2)
    elif scale_layout == "wide":
        big = torch.full(lead + (sr, 2 * ref.groups(cols) + 1), float("nan"), device=DEV)
        big[..., 1::2] = scale
        scale = big[..., 1::2]
    return data, scale


# ------------------------------------------------------------------------------ quantising

SHAPES = [(1, 1), (1, 128), (3, 127), (5, 129), (128, 128), (130, 260), (257, 1000), (64, 4096), (300, 520)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("along", ["rows", "columns", "blocks", "blocks_t"])
def test_quantize(along, rows, cols, dtype):
    x = numbers(rows, cols, rows * 7 + cols, dtype)
    if rows > 2:
        x[1] = 0                       # a row of zeros
    data, scale = tcl.quantize_fp8(x.to(DEV), along=along)
    source = x.t() if along == "columns" else x
    want, s = ref.quantize(source, 1 if along in ("rows", "columns") else 128)
    if along == "blocks_t":
        want, s = want.t(), s.t()
    assert torch.equal(scale.cpu(), s)
    assert torch.equal(data.cpu().double(), want)
    # and the values the pairs stand for are as near as e4m3 allows
    err = (ref.values(data, scale) - (source.t() if along == "blocks_t" else source).double()).abs()
    size = (source.t() if along == "blocks_t" else source).double().abs()
    assert bool((err <= torch.maximum(size * 2.0 ** -4, ref.widen(scale.cpu(), want.shape) * 2.0 ** -10) * (1 + 2.0 ** -20)).all())


def test_quantize_strided_unaligned_and_batched():
    big = numbers(40, 700, 5).to(DEV)
    for x in (big[:, 3:400], big[1::2, 8:648], big[:, :1], big[7:8, 5:300]):
        for along in ("rows", "columns", "blocks"):
            data, scale = tcl.quantize_fp8(x, along=along)
            want, s = ref.quantize(x.cpu().t() if along == "columns" else x.cpu(), 128 if along == "blocks" else 1)
            assert torch.equal(scale.cpu(), s) and torch.equal(data.cpu().double(), want)
    w = numbers(200, 300, 6, batch=5).to(DEV)
    for x in (w, w[::2], w[:, 10:50, 1:290], w[:0]):
        for along in ("blocks", "blocks_t"):
            data, scale = tcl.quantize_fp8(x, along=along)
            assert data.shape[0] == scale.shape[0] == x.shape[0]
            for i in range(x.shape[0]):
                want, s = ref.quantize(x[i].cpu(), 128)
                if along == "blocks_t":
                    want, s = want.t(), s.t()
                assert torch.equal(scale[i].cpu(), s) and torch.equal(data[i].cpu().double(), want)


def test_quantize_extremes():
    x = torch.zeros(8, 256)
    x[0, 3] = float("nan")
    x[1, 130] = float("inf")
    x[2, 5] = -float("inf")
    x[3] = 3.0e38
    x[4] = 1e-40                       # fp32 subnormals
    x[5, 1] = 2.0 ** -126
    x[6, :128] = -448.0
    x[6, 128:] = 1.0
    d, s = tcl.quantize_fp8(x.to(DEV))
    v = (d.float() * s.repeat_interleave(128, 1)).cpu()
    assert bool(torch.isnan(s[0, 0])) and bool(torch.isnan(v[0, :128]).all()) and bool((v[0, 128:] == 0).all())
    assert bool(torch.isinf(s[1, 1])) and bool(torch.isnan(v[1, 128:]).all()) and bool((v[1, :128] == 0).all())
    assert bool(torch.isnan(v[2, :128]).all())
    assert bool(((v[3] / 3.0e38 - 1).abs() < 1e-6).all())
    assert bool((v[4] - 1e-40).abs().max() <= 2.0 ** -126 * 2.0 ** -10)
    assert bool((v[6, :128] == -448).all()) and bool(((v[6, 128:] - 1).abs() < 1e-6).all())
    assert bool((d[7].float() == 0).all()) and bool((s[7] == 2.0 ** -126).all())
    dc, sc = tcl.quantize_fp8(x.to(DEV), along="columns")
    assert bool(torch.isnan(sc[3, 0])) and bool(torch.isnan(dc[3].float()).all())


def test_quantize_pads_rows_with_zeros():
    data, _ = tcl.quantize_fp8(numbers(9, 203, 3).to(DEV))
    full = data.as_strided((9, 208), (208, 1)).view(torch.uint8)
    assert bool((full[:, 203:] == 0).all())
    data, _ = tcl.quantize_fp8(numbers(203, 9, 3).to(DEV), along="columns")
    full = data.as_strided((9, 208), (208, 1)).view(torch.uint8)
    assert bool((full[:, 203:] == 0).all())


@pytest.mark.parametrize("along", ["rows", "columns"])
@pytest.mark.parametrize("tokens,top,experts,align,cols", [(1, 1, 1, 1, 64), (37, 3, 5, 1, 300), (50, 2, 4, 128, 257),
                                                           (200, 4, 16, 16, 512)])
def test_quantize_in_expert_order(along, tokens, top, experts, align, cols):
    g = torch.Generator().manual_seed(tokens)
    ids = torch.randint(-1, experts, (tokens, top), generator=g)
    x = numbers(tokens, cols, tokens + 1)
    order = tcl.sort_by_expert(ids.to(DEV), experts, align=align)
    data, scale = tcl.quantize_fp8(x.to(DEV), along=along, order=order)
    source = order.source.cpu().long()
    rows = x.float()[source.clamp_min(0) // top] * (source >= 0)[:, None]
    want, s = ref.quantize(rows.t() if along == "columns" else rows, 1)
    assert torch.equal(scale.cpu(), s)
    assert torch.equal(data.cpu().double(), want)


# ------------------------------------------------------------------------------ products

GEMMS = [(1, 1, 1), (1, 128, 128), (1, 4096, 1030), (2, 130, 300), (7, 100, 16), (16, 512, 2048), (17, 257, 129), (32, 640, 384),
         (33, 384, 513), (64, 200, 1000), (100, 776, 130), (128, 128, 128), (129, 129, 2000), (300, 1000, 640),
         (1000, 776, 1030), (600, 1000, 1024), (1024, 1536, 512), (1300, 2056, 259), (2000, 1111, 384), (70, 500, 4100),
         (130, 1000, 2050), (255, 300, 8192)]


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("per", [1, 128])
@pytest.mark.parametrize("M,N,K", GEMMS)
def test_gemm(M, N, K, per, out):
    pitch = -(-K // 16) * 16
    a, sa = random_operand(M, K, M + K, pitch=pitch)
    b, sb = random_operand(N, K, N + 2 * K, per=per, pitch=pitch)     # (what lies in the pitch is not zero)
    c = tcl.gemm_fp8(a, sa, b, sb, out_dtype=out)
    want, bound = ref.product_bound(ref.values(a, sa), ref.values(b, sb), out)
    ref.check(c, want, bound, f"{M}x{N}x{K}")


@pytest.mark.parametrize("M", [1, 20, 200])
def test_gemm_strides_and_alignment(M):
    N, K = 300, 400
    sa_kinds, pitches = ("groups", "rows", "wide"), (None, 416, 431)
    for i, layout in enumerate(sa_kinds):
        for pitch in pitches:
            a, sa = random_operand(M, K, 1 + i, pitch=pitch, scale_layout=layout)
            b, sb = random_operand(N, K, 2 + i, per=128 if i else 1, pitch=pitch, scale_layout=layout)
            want, bound = ref.product_bound(ref.values(a, sa), ref.values(b, sb), F32)
            ref.check(tcl.gemm_fp8(a, sa, b, sb, out_dtype=F32), want, bound, f"{layout} {pitch}")
    # bases off the 16-byte grid, and a result in the middle of a larger matrix
    a, sa = random_operand(M + 1, K + 3, 9, pitch=448)
    b, sb = random_operand(N + 1, K + 5, 10, pitch=448)
    a, b = a[1:, 3:], b[1:, 5:]
    sa, sb = sa[1:, :4].contiguous(), sb[1:, :4].contiguous()
    want, bound = ref.product_bound(ref.values(a, sa), ref.values(b, sb), BF16)
    for off in (0, 1, 8):
        big = torch.full((M + 2, N + 20), 7.0, dtype=BF16, device=DEV)
        c = big[1:M + 1, off:off + N]
        assert tcl.gemm_fp8(a, sa, b, sb, out=c) is c
        ref.check(c, want, bound, f"out at {off}")
        big[1:M + 1, off:off + N] = 7.0
        assert bool((big == 7.0).all())


def test_gemm_non_finite_values_stay_in_their_rows():
    for M in (4, 200):
        a, sa = random_operand(M, 256, 3)
        b, sb = random_operand(140, 256, 4)
        clean = tcl.gemm_fp8(a, sa, b, sb, out_dtype=F32)
        a.view(torch.uint8)[1, 200] = 0x7F
        sa[2, 0] = float("inf")
        b.view(torch.uint8)[130, 7] = 0xFF
        c = tcl.gemm_fp8(a, sa, b, sb, out_dtype=F32)
        assert bool(torch.isnan(c[1]).all()) and bool(torch.isnan(c[:, 130]).all())
        assert not bool(torch.isfinite(c[2]).any())
        keep = torch.ones_like(c, dtype=torch.bool)
        keep[1:3] = False
        keep[:, 130] = False
        assert torch.equal(c[keep], clean[keep])


@pytest.mark.parametrize("M,N,K", [(3, 200, 1), (40, 130, 131), (300, 300, 255), (1500, 1600, 140), (1500, 1600, 1030)])
def test_gemm_bytes_behind_a_row_do_not_count(M, N, K):
    pitch = -(-K // 16) * 16
    a, sa = random_operand(M, K, 3, pitch=pitch)
    b, sb = random_operand(N, K, 4, per=128, pitch=pitch)
    clean = tcl.gemm_fp8(a, sa, b, sb, out_dtype=F32)
    for t in (a, b):
        t.as_strided((t.shape[0], pitch), (pitch, 1)).view(torch.uint8)[:, K:] = 0x7F       # NaN
    assert torch.equal(tcl.gemm_fp8(a, sa, b, sb, out_dtype=F32), clean)
    want, bound = ref.product_bound(ref.values(a, sa), ref.values(b, sb), F32)
    ref.check(clean, want, bound)


def test_gemm_repeats_and_streams():
    a, sa = random_operand(513, 1024, 3)
    b, sb = random_operand(700, 1024, 4, per=128)
    c = tcl.gemm_fp8(a, sa, b, sb)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        assert torch.equal(tcl.gemm_fp8(a, sa, b, sb), c)
    d = tcl.gemm_fp8(a, sa, b, sb, stream=s)
    s.synchronize()
    assert torch.equal(c, d)


def test_streams_have_their_own_scratch():
    """Operands off the tensor copies' grid go through library scratch: calls on two streams at once."""
    jobs = []
    for i, (M, N, K) in enumerate([(900, 700, 1000), (5, 3000, 2000), (300, 300, 3001)]):
        a, sa = random_operand(M, K, 50 + i, pitch=K + 7)
        b, sb = random_operand(N, K, 60 + i, per=128, pitch=K + 5)
        jobs.append((a, sa, b, sb))
    want = [tcl.gemm_fp8(*job) for job in jobs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for turn in range(4):
        for k in range(3):
            for n, st in enumerate(streams):
                j = k if n == 0 else 2 - k
                got.append((j, tcl.gemm_fp8(*jobs[j], stream=st)))
    torch.cuda.synchronize()
    for j, c in got:
        assert torch.equal(c, want[j])
    for st in streams:
        tcl.stream_release(st)


def test_gemm_in_a_graph():
    x, w = numbers(100, 600, 1).to(DEV), numbers(300, 600, 2).to(DEV)
    wq, ws = tcl.quantize_fp8(w, along="blocks")
    want = tcl.gemm_fp8(*tcl.quantize_fp8(x), wq, ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = tcl.gemm_fp8(*tcl.quantize_fp8(x), wq, ws)
    got.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_gemm_no_rows():
    a, sa = random_operand(0, 256, 3)
    b, sb = random_operand(140, 256, 4)
    assert tcl.gemm_fp8(a, sa, b, sb).shape == (0, 140)


def test_gemm_past_32_bit_offsets():
    M, N, K = 530_000, 4096, 128         # C: 2.17e9 elements
    a, sa = random_operand(1000, K, 3)
    b, sb = random_operand(N, K, 4, per=128)
    small = tcl.gemm_fp8(a, sa, b, sb)
    c = tcl.gemm_fp8(a.view(torch.uint8).repeat(530, 1).view(F8), sa.repeat(530, 1), b, sb)
    assert torch.equal(c[-1000:], small) and torch.equal(c[:1000], small) and torch.equal(c[524_000:525_000], small)
    del c


# ------------------------------------------------------------------------------ experts

def offsets_of(counts, align=1):
    o = [0]
    for n in counts:
        o.append(o[-1] + -(-n // align) * align)
    return o


COUNTS = [[1], [0, 1, 0], [3, 0, 5, 1], [16, 17, 0, 15], [40, 1, 0, 33, 64], [130, 0, 127, 1, 256], [0, 0, 700, 0], [300] * 5, [700, 513, 0, 1025]]


@pytest.mark.parametrize("N,K,per,out", [(128, 128, 128, BF16), (300, 513, 128, F32), (257, 640, 1, BF16), (1, 16, 1, F32), (1000, 200, 128, BF16)])
@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("behind", [0, 3, 200])
def test_experts(counts, N, K, per, out, behind):
    o = offsets_of(counts)
    rows, E = o[-1] + behind, len(counts)
    a, sa = random_operand(rows, K, rows + K, pitch=-(-K // 16) * 16)
    b, sb = random_operand(N, K, N + K, per=per, pitch=-(-K // 16) * 16, batch=E)
    c = tcl.gemm_fp8_experts(a, sa, b, sb, torch.tensor(o, dtype=torch.int32, device=DEV), out_dtype=out)
    va, vb = ref.values(a, sa), ref.values(b, sb)
    for e in range(E):
        want, bound = ref.product_bound(va[o[e]:o[e + 1]], vb[e], out)
        ref.check(c[o[e]:o[e + 1]], want, bound, f"expert {e}")
    assert bool((c[o[-1]:] == 0).all())


def test_experts_strides():
    o = [0, 5, 5, 40]
    a, sa = random_operand(40, 200, 1, pitch=205, scale_layout="wide")
    b, sb = random_operand(100, 200, 2, per=128, batch=6, pitch=203, scale_layout="wide")
    b, sb = b[::2], sb[::2]
    c = tcl.gemm_fp8_experts(a, sa, b, sb, torch.tensor(o, dtype=torch.int32, device=DEV), out_dtype=F32)
    va, vb = ref.values(a, sa), ref.values(b, sb)
    for e in range(3):
        want, bound = ref.product_bound(va[o[e]:o[e + 1]], vb[e], F32)
        ref.check(c[o[e]:o[e + 1]], want, bound, f"expert {e}")


def test_many_experts():
    E, N, K = 1000, 64, 128
    g = torch.Generator().manual_seed(5)
    counts = torch.randint(0, 5, (E,), generator=g).tolist()
    o = offsets_of(counts)
    a, sa = random_operand(o[-1], K, 1)
    b, sb = random_operand(N, K, 2, per=128, batch=E)
    c = tcl.gemm_fp8_experts(a, sa, b, sb, torch.tensor(o, dtype=torch.int32, device=DEV), out_dtype=F32)
    va, vb = ref.values(a, sa), ref.values(b, sb)
    for e in range(E):
        want, bound = ref.product_bound(va[o[e]:o[e + 1]], vb[e], F32)
        ref.check(c[o[e]:o[e + 1]], want, bound, f"expert {e}")


@pytest.mark.parametrize("o,rows", [([0, 5, 3, 10], 10), ([1, 5, 8, 10], 10), ([0, 5, 8, 11], 10), ([0, -1, 8, 10], 10)])
def test_bad_offsets_are_reported(o, rows):
    a, sa = random_operand(rows, 128, 1)
    b, sb = random_operand(64, 128, 2, per=128, batch=3)
    out = torch.full((rows, 64), 5.0, dtype=F32, device=DEV)
    tcl.gemm_fp8_experts(a, sa, b, sb, torch.tensor(o, dtype=torch.int32, device=DEV), out=out)
    assert tcl.last_device_error() == (7, 7)
    assert bool((out == 5.0).all())
    assert tcl.last_device_error() == (0, 0)


@pytest.mark.parametrize("N,K,out", [(128, 128, F32), (300, 77, F32), (64, 513, BF16), (1, 1, F32), (1000, 900, F32),
                                     (1024, 1281, BF16)])
@pytest.mark.parametrize("counts", [[1], [0, 3], [128, 0, 0, 300], [5, 640, 130, 0, 1]])
@pytest.mark.parametrize("behind", [0, 128, 40])
def test_wgrad(counts, N, K, out, behind):
    o = offsets_of(counts, 128)
    rows, E = o[-1] + behind, len(counts)
    pitch = -(-rows // 16) * 16
    a, sa = random_operand(N, rows, N + rows, pitch=pitch)
    b, sb = random_operand(K, rows, K + 3 * rows, pitch=pitch)
    c = tcl.gemm_fp8_experts_wgrad(a, sa, b, sb, torch.tensor(o, dtype=torch.int32, device=DEV), out_dtype=out)
    assert c.shape == (E, N, K)
    va, vb = ref.values(a, sa), ref.values(b, sb)
    for e in range(E):
        want, bound = ref.product_bound(va[:, o[e]:o[e + 1]], vb[:, o[e]:o[e + 1]], out)
        ref.check(c[e], want, bound, f"expert {e}")


@pytest.mark.parametrize("counts", [[9000], [5000, 0, 130, 4000]])
def test_wgrad_of_many_rows_and_few_tiles(counts):
    """Clusters share the rows of a tile, unevenly long experts and empty ones among them."""
    o = offsets_of(counts, 128)
    E, N, K = len(counts), 200, 130
    a, sa = random_operand(N, o[-1], 1)
    b, sb = random_operand(K, o[-1], 2)
    c = tcl.gemm_fp8_experts_wgrad(a, sa, b, sb, torch.tensor(o, dtype=torch.int32, device=DEV), out_dtype=F32)
    va, vb = ref.values(a, sa), ref.values(b, sb)
    for e in range(E):
        want, bound = ref.product_bound(va[:, o[e]:o[e + 1]], vb[:, o[e]:o[e + 1]], F32)
        ref.check(c[e], want, bound, f"expert {e}")


def test_wgrad_refuses_offsets_off_the_groups():
    a, sa = random_operand(64, 256, 1)
    b, sb = random_operand(64, 256, 2)
    tcl.gemm_fp8_experts_wgrad(a, sa, b, sb, torch.tensor([0, 100, 256], dtype=torch.int32, device=DEV))
    assert tcl.last_device_error() == (7, 7)


def test_wgrad_no_rows():
    z, s = torch.empty(64, 0, dtype=F8, device=DEV), torch.empty(64, 0, device=DEV)
    c = tcl.gemm_fp8_experts_wgrad(z, s, z, s, torch.zeros(4, dtype=torch.int32, device=DEV))
    assert c.shape == (3, 64, 64) and bool((c == 0).all())


def test_wgrad_against_differences():
    """L(W) = sum of G·(X·Wᵀ) is linear in each W[e], so a difference quotient is exact in 64 bits."""
    o = [0, 128, 128, 384]
    x, dy = numbers(384, 96, 1), numbers(384, 80, 2)
    xq, xs = tcl.quantize_fp8(x.to(DEV), along="columns")
    gq, gs = tcl.quantize_fp8(dy.to(DEV), along="columns")
    dw = tcl.gemm_fp8_experts_wgrad(gq, gs, xq, xs, torch.tensor(o, dtype=torch.int32, device=DEV), out_dtype=F32)
    vx, vg = ref.values(xq, xs).t(), ref.values(gq, gs).t()
    g = torch.Generator().manual_seed(3)

    def loss(w):
        return sum(float((vg[i:j] * (vx[i:j] @ w[e].t())).sum()) for e, (i, j) in enumerate(zip(o, o[1:])))

    for _ in range(4):
        w, d = torch.randn(3, 80, 96, generator=g).double(), torch.randn(3, 80, 96, generator=g).double()
        slope = (loss(w + d) - loss(w - d)) / 2
        # the quotient's sum differs by no more than each element's own bound, weighted
        near = sum(float((ref.product_bound(vg[i:j].t(), vx[i:j].t(), F32)[1] * d[e].abs()).sum())
                   for e, (i, j) in enumerate(zip(o, o[1:])))
        assert abs(float((dw.cpu().double() * d).sum()) - slope) <= near + 1e-9 * abs(slope)
