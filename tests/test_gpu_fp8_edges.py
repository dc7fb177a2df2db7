"""Edges of the e4m3 quantising, products and routing on the GPU: padding beside non-finite values,
captures, threads, sizes past the grid's axes, pair tiles over several waves, operands off the
tensor copies' grid."""
from __future__ import annotations

import pytest
import torch

import fp8_reference as ref
import tensor_core_loop_gb300 as tcl
from tensor_core_loop_gb300 import fp8

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


def random_operand(rows, cols, seed, per=1, pitch=None, batch=None, distance=None):
    """e4m3 data of any bit pattern but NaN, with scales over a few powers of two; rows `pitch` bytes and
    matrices `distance` bytes apart."""
    g = torch.Generator().manual_seed(seed)
    pitch = pitch or cols
    distance = distance or rows * pitch
    bits = torch.randint(0, 254, ((batch or 1) * distance,), generator=g, dtype=torch.uint8)
    data = torch.where(bits >= 127, bits + 1, bits).view(F8).to(DEV)     # (0x7f and 0xff are NaN)
    lead = () if batch is None else (batch,)
    data = data.as_strided(lead + (rows, cols), (distance, pitch, 1)[1 - len(lead):])
    scale = torch.exp2(3 * torch.randn(lead + (-(-rows // per), ref.groups(cols)), generator=g)).to(DEV)
    return data, scale


# ------------------------------------------------------------------------------ quantising

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("along", ["rows", "columns", "blocks", "blocks_t", "rows in order", "columns in order"])
def test_padding_is_zero_beside_non_finite_values(along, value, dtype):
    """The bytes between a row's end and the next multiple of 16 are zeros whatever the last group holds."""
    x = torch.randn(140, 203, generator=torch.Generator().manual_seed(1)).to(dtype)
    x[139, 202] = value
    x[0, 202] = value
    x[139, 0] = value
    order = None
    if "order" in along:
        order = tcl.sort_by_expert(torch.zeros(140, 1, dtype=torch.int32, device=DEV), 1)
    data, scale = tcl.quantize_fp8(x.to(DEV), along=along.split()[0], order=order)
    rows, cols = data.shape
    pitch = -(-cols // 16) * 16
    assert pitch > cols and data.stride(0) == pitch
    padding = data.as_strided((rows, pitch), (pitch, 1)).view(torch.uint8)[:, cols:]
    assert bool((padding == 0).all())
    assert not bool(torch.isfinite(scale).all())      # (and the groups that hold the value carry it)


@pytest.mark.parametrize("along", ["columns", "blocks", "blocks_t"])
def test_more_tiles_than_a_grid_axis_holds(along):
    """65,536 tiles of 128 rows and a piece, and 65,537 matrices of a batch."""
    cut, rows = 65_535 * 128, 65_536 * 128 + 5
    x = torch.randn(rows, 3, device=DEV, generator=torch.Generator(device=DEV).manual_seed(2)).to(BF16)
    data, scale = tcl.quantize_fp8(x, along=along)
    tail = x[cut:].cpu()
    want, s = ref.quantize(tail.t() if along == "columns" else tail, 1 if along == "columns" else 128)
    if along == "blocks":
        assert torch.equal(data[cut:].cpu().double(), want) and torch.equal(scale[cut // 128:].cpu(), s)
    else:
        want, s = (want, s) if along == "columns" else (want.t(), s.t())
        assert torch.equal(data[:, cut:].cpu().double(), want) and torch.equal(scale[:, cut // 128:].cpu(), s)
    head = tcl.quantize_fp8(x[:cut], along=along)      # (as many as fit the axis)
    got = (data[:cut], scale[:cut // 128]) if along == "blocks" else (data[:, :cut], scale[:, :cut // 128])
    assert torch.equal(got[0].float(), head[0].float()) and torch.equal(got[1], head[1])
    if along != "blocks":      # rows of the result that leave no room behind them
        tight, st = torch.empty(3, rows, dtype=F8, device=DEV), torch.empty_like(scale)
        if along == "columns":
            status = fp8._lib().tcl_quantize_fp8_columns(0, rows, 3, x.data_ptr(), 3, None, 1, 0, tight.data_ptr(), rows,
                                                         st.data_ptr(), *st.stride(), torch.cuda.current_stream().cuda_stream)
        else:
            status = fp8._lib().tcl_quantize_fp8_blocks(0, 1, rows, 3, x.data_ptr(), 3, 0, 1, tight.data_ptr(), rows, 0,
                                                        st.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert status == 0 and torch.equal(tight.view(torch.uint8), data.view(torch.uint8)) and torch.equal(st, scale)
    if along != "columns":
        w = torch.randn(65_537, 2, 3, device=DEV, generator=torch.Generator(device=DEV).manual_seed(3))
        data, scale = tcl.quantize_fp8(w, along=along)
        top = w.abs().amax((1, 2))
        v = (data.float() * scale).double()
        v = v.transpose(1, 2) if along == "blocks_t" else v
        assert bool(((v - w.double()).abs() <= top[:, None, None].double() * 2.0 ** -4).all())
        assert torch.equal(scale.view(-1), torch.div(top, torch.full_like(top, 448.0)))


# ------------------------------------------------------------------------------ sorting

def test_sort_of_many_slots_in_a_graph():
    """Captured on a stream that the library has not seen, with no scratch in place, and replayed
    beside sorts on the default stream."""
    E, shape = 500, (30_000, 4)
    g = torch.Generator().manual_seed(4)
    first, second, third = (torch.randint(-1, E, shape, generator=g) for _ in range(3))
    ids, others = first.to(DEV), third.to(DEV)
    torch.cuda.synchronize()
    tcl.lib().tcl_shutdown()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = tcl.sort_by_expert(ids, E, align=16)
    ids.copy_(second)
    torch.cuda.synchronize()
    side, beside = torch.cuda.Stream(), []
    with torch.cuda.stream(side):
        for _ in range(20):
            graph.replay()
    for _ in range(20):
        beside.append(tcl.sort_by_expert(others, E, align=16))
    torch.cuda.synchronize()
    for order, of in ((got, second), *((b, third) for b in beside[::7])):
        offsets, position, source = ref.order(of, E, 16, order.source.numel())
        assert order.offsets.tolist() == offsets
        assert order.position.reshape(-1).tolist() == position and order.source.tolist() == source


@pytest.mark.parametrize("tokens,top,experts,align", [(4097, 1, 1024, 1), (4097, 1, 1024, 128), (1366, 3, 1023, 2), (8193, 1, 33, 128),
                                                      (2731, 3, 1024, 128), (40_000, 7, 100, 3), (12_289, 1, 1, 128)])
def test_sort_just_past_a_block(tokens, top, experts, align):
    g = torch.Generator().manual_seed(tokens)
    ids = torch.randint(-1, experts, (tokens, top), generator=g)
    for of in (ids, torch.full_like(ids, -1), torch.full_like(ids, experts - 1)):
        got = tcl.sort_by_expert(of.to(DEV), experts, align=align)
        offsets, position, source = ref.order(of, experts, align, got.source.numel())
        assert got.offsets.tolist() == offsets
        assert got.position.reshape(-1).tolist() == position and got.source.tolist() == source


def test_sort_of_millions_of_slots():
    tokens, top, E, align = 600_001, 7, 200, 128
    ids = torch.randint(-1, E, (tokens, top), device=DEV, generator=torch.Generator(device=DEV).manual_seed(6))
    offsets, position, source = tcl.sort_by_expert(ids, E, align=align)
    flat = ids.reshape(-1)
    count = torch.bincount(flat[flat >= 0], minlength=E)
    length = (count + align - 1) // align * align
    want = torch.nn.functional.pad(length.cumsum(0), (1, 0))
    assert torch.equal(offsets.long(), want)
    slots = torch.argsort(torch.where(flat >= 0, flat, E), stable=True)[:int(count.sum())]
    e = flat[slots]
    row = want[e] + torch.arange(len(slots), device=DEV) - torch.nn.functional.pad(count.cumsum(0), (1, 0))[e]
    assert torch.equal(position.view(-1)[slots].long(), row) and bool((position.view(-1)[flat < 0] == -1).all())
    full = torch.full_like(source, -1)
    full[row] = slots.int()
    assert torch.equal(source, full)


# ------------------------------------------------------------------------------ streams and threads

def test_operands_of_another_streams_call_are_kept():
    """Memory of an operand that is dropped right after the call is not handed out while the given
    stream may still read it."""
    s = torch.cuda.Stream()
    x = torch.randn(600, 512, device=DEV).to(BF16)
    a, sa = tcl.quantize_fp8(x)
    b, sb = tcl.quantize_fp8(x, along="blocks")
    want = tcl.gemm_fp8(a, sa, b, sb)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)                  # (a tenth of a second)
    c = tcl.gemm_fp8(a, sa, b, sb, stream=s)
    kept = {t.data_ptr() for t in (a, sa, b, sb)}
    like = [(t.shape, t.stride(), t.dtype) for t in (a, sa, b, sb)]
    del a, sa, b, sb
    again = [torch.empty_strided(size, stride, dtype=dtype, device=DEV) for size, stride, dtype in like]
    assert not kept & {t.data_ptr() for t in again}
    s.synchronize()
    assert torch.equal(c, want)


def test_threads_on_one_stream():
    """Calls of several launches from several threads (ctypes lets the others run meanwhile): products whose
    operands go through library scratch, and sorts."""
    from concurrent.futures import ThreadPoolExecutor
    jobs = []
    for i, (M, N, K) in enumerate([(200, 300, 500), (700, 300, 900), (90, 2000, 1200), (1000, 600, 260)]):
        a, sa = random_operand(M, K, 70 + i, pitch=K + 7)
        b, sb = random_operand(N, K, 80 + i, per=128, pitch=K + 5)
        ids = torch.randint(0, 40 * (i + 1), (2000 * (i + 2), 3), generator=torch.Generator().manual_seed(i)).to(DEV)
        jobs.append((a, sa, b, sb, ids, 40 * (i + 1)))

    def turn(job):
        a, sa, b, sb, ids, E = job
        return tcl.gemm_fp8(a, sa, b, sb), *tcl.sort_by_expert(ids, E, align=8)

    want = [turn(job) for job in jobs]
    torch.cuda.synchronize()
    with ThreadPoolExecutor(4) as pool:
        got = [r for r in pool.map(lambda i: (i % 4, turn(jobs[i % 4])), range(400))]
    torch.cuda.synchronize()
    for i, r in got:
        for u, v in zip(r, want[i]):
            assert torch.equal(u, v)


# ------------------------------------------------------------------------------ products

def test_gemm_of_a_row_past_half_of_32_bits():
    """More than 2^30 values of K in operands that are copied onto the tensor copies' grid first."""
    K = 2 ** 30 + 300
    a, b = (torch.zeros(K + 1, dtype=torch.uint8, device=DEV) for _ in range(2))
    at = torch.tensor([0, 5, 127, 128, 2 ** 29 + 1, 2 ** 30 - 1, 2 ** 30, 2 ** 30 + 257, K - 1], device=DEV) + 1
    a[at], b[at] = 0x38, 0x40                            # 1 and 2
    one = torch.ones(1, device=DEV).expand(1, -(-K // 128))
    c = tcl.gemm_fp8(a.view(F8)[None, 1:], one, b.view(F8)[None, 1:], one, out_dtype=F32)
    assert float(c) == 2.0 * len(at)
    torch.cuda.synchronize()
    tcl.lib().tcl_shutdown()                             # (2 GB of scratch)


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def pair_tiles(counts, N, experts):
    """Tiles of 256 x 256 that rows sorted by expert make, if that is the tile that the library takes for
    them (from some hundred rows an expert, where tiles of 128 x 128 are more than the SMs)."""
    rows = sum(counts)
    each = -(-rows // experts)
    ones = -(-each // 128) * -(-N // 128) * experts
    return sum(-(-n // 256) for n in counts) * -(-N // 256) if each > 112 and N > 128 and ones > sms() else 0


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("per", [1, 128])
@pytest.mark.parametrize("M,N,K", [(3000, 2600, 1300), (3001, 2601, 1153), (2817, 2304, 2048)])
def test_gemm_pair_tiles_over_several_waves(M, N, K, per, out):
    """Every pair of SMs walks more than one tile of more than eight k-blocks: the rings' phases, the scales'
    slots and the slabs of the stores go on from one tile to the next."""
    assert pair_tiles([M], N, 1) > sms() // 2 and K > 8 * 128
    pitch = -(-K // 16) * 16
    a, sa = random_operand(M, K, M + K, pitch=pitch)
    b, sb = random_operand(N, K, N + 2 * K, per=per, pitch=pitch)
    c = tcl.gemm_fp8(a, sa, b, sb, out_dtype=out)
    want, bound = ref.product_bound(ref.values(a, sa), ref.values(b, sb), out)
    ref.check(c, want, bound, f"{M}x{N}x{K}")


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("per", [1, 128])
@pytest.mark.parametrize("N,K", [(1100, 1300), (1111, 1300), (1280, 1153)])
@pytest.mark.parametrize("behind", [0, 300])
def test_experts_pair_tiles_over_several_waves(N, K, per, out, behind):
    counts = [2300, 0, 513, 1, 1700, 0, 260, 1226]
    assert pair_tiles(counts + [behind], N, len(counts)) > sms() // 2 and K > 8 * 128
    o = [sum(counts[:i]) for i in range(len(counts) + 1)]
    rows, E, pitch = o[-1] + behind, len(counts), -(-K // 16) * 16
    a, sa = random_operand(rows, K, rows + K, pitch=pitch)
    b, sb = random_operand(N, K, N + K, per=per, pitch=pitch, batch=E)
    c = tcl.gemm_fp8_experts(a, sa, b, sb, torch.tensor(o, dtype=torch.int32, device=DEV), out_dtype=out)
    va, vb = ref.values(a, sa), ref.values(b, sb)
    for e in range(E):
        want, bound = ref.product_bound(va[o[e]:o[e + 1]], vb[e], out)
        ref.check(c[o[e]:o[e + 1]], want, bound, f"expert {e}")
    assert bool((c[o[-1]:] == 0).all())


# (rows of operands and results off the tensor copies' grid, matrices at odd distances, strided scales)

def strided(scale):
    """The same scales, every second column of a larger matrix, NaN between them."""
    big = torch.full((*scale.shape[:-1], 2 * scale.shape[-1] + 1), float("nan"), device=DEV)
    big[..., 1::2] = scale
    return big[..., 1::2]


@pytest.mark.parametrize("counts", [[3, 0, 5, 1], [130, 0, 127, 300], [700, 513, 0, 1025]])
@pytest.mark.parametrize("pitch,distance", [(208, 300 * 208 + 1), (208, 300 * 208 + 8), (207, 300 * 207 + 3), (208, 301 * 208)])
def test_experts_matrices_at_any_distance(counts, pitch, distance):
    """An aligned base and leading dimension with the matrices off the grid: all of them are copied."""
    N, K, E = 300, 200, len(counts)
    o = [sum(counts[:i]) for i in range(E + 1)]
    a, sa = random_operand(o[-1], K, 1, pitch=208)
    b, sb = random_operand(N, K, 2, per=128, pitch=pitch, batch=E, distance=distance)
    c = tcl.gemm_fp8_experts(a, strided(sa), b, strided(sb), torch.tensor(o, dtype=torch.int32, device=DEV), out_dtype=F32)
    va, vb = ref.values(a, sa), ref.values(b, sb)
    for e in range(E):
        want, bound = ref.product_bound(va[o[e]:o[e + 1]], vb[e], F32)
        ref.check(c[o[e]:o[e + 1]], want, bound, f"expert {e}")


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("counts", [[2, 1], [60, 33], [3000, 1500, 0, 2001]])
@pytest.mark.parametrize("off", [0, 1, 8])
def test_experts_into_a_part_of_a_matrix(counts, off, out):
    N, K, E = 700, 300, len(counts)
    o = [sum(counts[:i]) for i in range(E + 1)]
    rows = o[-1] + 5
    a, sa = random_operand(rows, K, 1, pitch=304)
    b, sb = random_operand(N, K, 2, per=128, pitch=304, batch=E)
    big = torch.full((rows + 2, N + 20), 7.0, dtype=out, device=DEV)
    c = big[1:rows + 1, off:off + N]
    assert tcl.gemm_fp8_experts(a, sa, b, sb, torch.tensor(o, dtype=torch.int32, device=DEV), out=c) is c
    va, vb = ref.values(a, sa), ref.values(b, sb)
    for e in range(E):
        want, bound = ref.product_bound(va[o[e]:o[e + 1]], vb[e], out)
        ref.check(c[o[e]:o[e + 1]], want, bound, f"expert {e}")
    assert bool((c[o[-1]:] == 0).all())
    c.fill_(7.0)
    assert bool((big == 7.0).all())


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("N,K,counts", [(130, 77, [5, 300, 0]), (64, 300, [4000, 1]), (1030, 1100, [256, 0, 900, 130] * 4)])
@pytest.mark.parametrize("pitches,off", [((None, None), 0), ((3, 16), 1), ((16, 5), 8), ((1, 7), 16)])
def test_wgrad_strides_and_alignment(N, K, counts, out, pitches, off):
    """Operands at any pitch, strided scales, the result in the middle of a larger batch."""
    o = [0]
    for n in counts:
        o.append(o[-1] + -(-n // 128) * 128)
    rows, E = o[-1], len(counts)
    a, sa = random_operand(N, rows, 1, pitch=rows + pitches[0] if pitches[0] else None)
    b, sb = random_operand(K, rows, 2, pitch=rows + pitches[1] if pitches[1] else None)
    big = torch.full((E, N + 2, K + 24), 7.0, dtype=out, device=DEV)
    c = big[:, 1:N + 1, off:off + K]
    assert tcl.gemm_fp8_experts_wgrad(a, strided(sa), b, strided(sb), torch.tensor(o, dtype=torch.int32, device=DEV), out=c) is c
    va, vb = ref.values(a, sa), ref.values(b, sb)
    for e in range(E):
        want, bound = ref.product_bound(va[:, o[e]:o[e + 1]], vb[:, o[e]:o[e + 1]], out)
        ref.check(c[e], want, bound, f"expert {e}")
    c.fill_(7.0)
    assert bool((big == 7.0).all())
