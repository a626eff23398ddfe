"""The grouped int8 product and the SwiGLU FFN made of it, against exact integer sums
(the products bit for bit) and 64 bits (int8_reference.py has the FFN's bounds)."""
import pytest
import torch

import combine_moe_route_03_amd as moe
import int8_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
I32 = dict(dtype=torch.int32, device=DEV)


def ints(*shape, seed, low=-127, high=127):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(low, high + 1, shape, generator=g, device=DEV, dtype=torch.int32).to(torch.int8)


def scales(*shape, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.exp(torch.randn(shape, generator=g, device=DEV)) * 0.01


def buckets(counts, gap=0):
    """Offsets of buckets laid side by side, `gap` rows between them."""
    offs, at = [], 0
    for n in counts:
        offs.append(at)
        at += n + gap
    return torch.tensor(offs, **I32), torch.tensor(counts, **I32), at


def check(a, sa, offs, cnts, w, sw, index=None, rows=None, dtype=torch.bfloat16):
    rows = (a.shape[0] if index is None else index.numel()) if rows is None else rows
    out = torch.full((rows, w.shape[1]), 77.0, device=DEV, dtype=dtype)
    want = ref.gemm(a, sa, offs, cnts, w, sw, index, out.clone())
    got = moe.expert_gemm_int8(a, sa, offs, cnts, w, sw, row_token=index, out=out)
    assert got is out
    bad = (out != want).any(1).nonzero().flatten().tolist()
    assert not bad, f"rows {bad[:8]} of {rows}, columns {(out != want).any(0).nonzero().flatten().tolist()[:8]}"


# rows of the experts: none, one, around 8, 16, 32 and 256, and far more
COUNTS = [[0], [1], [7, 0, 1], [8, 9], [16, 17, 31], [32, 33, 1, 0, 64, 65], [100, 3], [255, 256, 257],
          [29, 300, 0, 0, 513], [700]]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("N,K", [(16, 16), (48, 128), (272, 144), (512, 400), (1040, 1408)])
def test_gemm(N, K, counts, dtype):
    print(f"[gemm int8] N={N} K={K} counts={counts} {dtype}", flush=True)
    offs, cnts, rows = buckets(counts)
    E = len(counts)
    check(ints(rows, K, seed=1), scales(rows, seed=2), offs, cnts, ints(E, N, K, seed=3),
          scales(E, N, seed=4), dtype=dtype)


@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("N,K", [(16, 48), (272, 144), (512, 512), (800, 4096)])
def test_gemm_rows_by_index(N, K, counts):
    """Rows picked from tokens, one token for several rows, indexes outside the tokens."""
    print(f"[gemm int8] N={N} K={K} counts={counts} by index", flush=True)
    offs, cnts, rows = buckets(counts)
    E, T = len(counts), 37
    g = torch.Generator(device=DEV).manual_seed(5)
    index = torch.randint(0, T, (rows,), generator=g, device=DEV, dtype=torch.int32)
    for i, bad in enumerate((-1, T, 2 ** 31 - 1, -2 ** 31, 1 << 28)):
        if rows > 3 * i + 1:
            index[3 * i + 1] = bad
    check(ints(T, K, seed=6), scales(T, seed=7), offs, cnts, ints(E, N, K, seed=8),
          scales(E, N, seed=9), index=index)


@pytest.mark.parametrize("rows,K", [(1, 64), (20, 400), (40, 64), (40, 400), (300, 1040)])
def test_gemm_no_tokens(rows, K):
    """Rows by index into no tokens are rows of zeros."""
    index = torch.zeros(rows, **I32)
    a, sa = torch.empty(0, K, device=DEV, dtype=torch.int8), torch.empty(0, device=DEV)
    out = moe.expert_gemm_int8(a, sa, torch.tensor([0], **I32), torch.tensor([rows], **I32),
                               ints(1, 32, K, seed=1), scales(1, 32, seed=2), row_token=index)
    assert (out == 0).all()


# more than 14 or 28 rows an expert and 2^20 results: the tiled kernel, tiles of 1 to 256 rows;
# of up to 128 where there are few tiles or rows an expert and more than two K steps
TILED = [[700], [255, 256, 257, 64, 65, 128, 129, 1, 0, 300], [1, 1999, 0], [513, 30, 31, 32, 33, 511],
         [2047, 1, 897, 95, 0, 160], [33] * 40 + [127, 0, 31, 3], [16, 0, 33, 1, 17, 96, 5, 18] * 8]


def tiled(rows, E, N, K):
    return K > 128 and rows > (8 if K % 128 else 14 if K < 4096 else 28) * E and (rows + 16 * min(rows, E)) * N > 2 ** 20 + 16 * N


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts", TILED, ids=str)
@pytest.mark.parametrize("N,K", [(4112, 144), (4096, 256), (3600, 272), (4368, 1408), (8208, 400),
                                 (2064, 528)])
def test_gemm_tiled(N, K, counts, dtype):
    print(f"[gemm int8 tiled] N={N} K={K} counts={counts} {dtype}", flush=True)
    offs, cnts, rows = buckets(counts)
    E = len(counts)
    assert tiled(rows, E, N, K)
    w, sw = ints(E, N, K, seed=3), scales(E, N, seed=4)
    check(ints(rows, K, seed=1), scales(rows, seed=2), offs, cnts, w, sw, dtype=dtype)
    index = torch.randint(0, 37, (rows,), generator=torch.Generator(device=DEV).manual_seed(5),
                          device=DEV, dtype=torch.int32)
    for i, bad in enumerate((-1, 37, 2 ** 31 - 1, -2 ** 31, 1 << 28)):
        index[rows // 5 * i + 1] = bad
    check(ints(37, K, seed=6), scales(37, seed=7), offs, cnts, w, sw, index=index, dtype=dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts", [[1], [5], [8], [9], [17], [32], [33], [1, 0, 2], [0, 40, 3, 8]], ids=str)
@pytest.mark.parametrize("N,K", [(16, 1040), (48, 7168), (1040, 2064), (2064, 1536), (4112, 4096)])
def test_gemm_few_columns(N, K, counts, dtype):
    """Few tiles: every wave of a block a part of K, groups of 16 columns and of 32."""
    offs, cnts, rows = buckets(counts)
    E = len(counts)
    check(ints(rows, K, seed=1), scales(rows, seed=2), offs, cnts, ints(E, N, K, seed=3),
          scales(E, N, seed=4), dtype=dtype)


@pytest.mark.parametrize("rows", [900, 4000])
def test_gemm_tiled_no_tokens(rows):
    index = torch.zeros(rows, **I32)
    a, sa = torch.empty(0, 1040, device=DEV, dtype=torch.int8), torch.empty(0, device=DEV)
    out = moe.expert_gemm_int8(a, sa, torch.tensor([0], **I32), torch.tensor([rows], **I32),
                               ints(1, 4096, 1040, seed=1), scales(1, 4096, seed=2), row_token=index)
    assert tiled(rows, 1, 4096, 1040) and (out == 0).all()


def test_gemm_tiled_rounds():
    """More tiles than compute units, with a rest that is cut; rows of all sizes."""
    g = torch.Generator().manual_seed(1)
    for E, N, K, most in ((70, 4096, 272, 300), (5, 8208, 400, 2500), (300, 2064, 144, 130),
                          (6, 8208, 2064, 2500), (40, 4112, 2304, 400)):
        counts = torch.randint(0, most, (E,), generator=g).tolist()
        offs, cnts, rows = buckets(counts)
        assert tiled(rows, E, N, K)
        check(ints(rows, K, seed=1), scales(rows, seed=2), offs, cnts, ints(E, N, K, seed=3),
              scales(E, N, seed=4))


@pytest.mark.parametrize("rows", [600, 3000])
def test_gemm_tiled_largest_sums(rows):
    """The longest K, every product the largest, through the tiled kernel."""
    N, K = 4096, 131056
    assert tiled(rows, 1, N, K)
    w = torch.full((1, N, K), -128, device=DEV, dtype=torch.int8)
    w[0, ::2] = 127
    offs, cnts, _ = buckets([rows])
    out = moe.expert_gemm_int8(torch.full((rows, K), -128, device=DEV, dtype=torch.int8),
                               torch.ones(rows, device=DEV), offs, cnts, w,
                               torch.ones(1, N, device=DEV), out_dtype=torch.float32)
    assert (out[:, 1::2] == 16384.0 * K).all() and (out[:, ::2] == -16256.0 * K).all()


@pytest.mark.parametrize("N,rows_each", [(144, 5), (144, 60), (144, 300), (2064, 300)])
def test_gemm_buckets(N, rows_each):
    """Buckets in another order with rows between them; buckets that leave the rows or
    have no sense give nothing; rows in no bucket stay as they were."""
    n = rows_each
    E, K = 9, 272
    rows = 5 * n + 40
    offs = [3 * n + 21, 0, 2 * n + 9, rows - n, -1, rows - n + 1, 0, 2 ** 31 - 1, n + 2]
    cnts = [n, n, n - 1, n, n, n, -4, 2 ** 31 - 1, n - 3]
    check(ints(rows, K, seed=1), scales(rows, seed=2), torch.tensor(offs, **I32),
          torch.tensor(cnts, **I32), ints(E, N, K, seed=3), scales(E, N, seed=4))


@pytest.mark.parametrize("E", [65, 300, 1024])
def test_gemm_many_experts(E):
    g = torch.Generator().manual_seed(E)
    for most in (2, 40):
        counts = torch.randint(0, most, (E,), generator=g).tolist()
        offs, cnts, rows = buckets(counts)
        check(ints(rows, 256, seed=1), scales(rows, seed=2), offs, cnts, ints(E, 80, 256, seed=3),
              scales(E, 80, seed=4))


@pytest.mark.parametrize("rows", [3, 40, 300])
def test_gemm_largest_sums(rows):
    """The longest K with every product the largest: sums next to 2^31, both signs."""
    K = 131056
    a = torch.full((rows, K), -128, device=DEV, dtype=torch.int8)
    w = torch.full((1, 32, K), -128, device=DEV, dtype=torch.int8)
    w[0, 16:] = 127
    offs, cnts, _ = buckets([rows])
    check(a, torch.full((rows,), 1.0, device=DEV), offs, cnts, w, torch.ones(1, 32, device=DEV),
          dtype=torch.float32)


def test_gemm_scales_at_the_ends():
    """Scales of any size, zero, infinite and NaN: what fp32 makes of them."""
    N, K = 48, 144
    for rows in (9, 300):
        sa, sw = scales(rows, seed=1), scales(1, N, seed=2)
        sa[0], sa[1], sa[2], sa[3] = 1e30, 1e-38, float("nan"), 0
        sw[0, 1], sw[0, 2], sw[0, 5] = 1e-30, 3e38, float("inf")
        offs, cnts, _ = buckets([rows])
        a, w = ints(rows, K, seed=3), ints(1, N, K, seed=4)
        out = moe.expert_gemm_int8(a, sa, offs, cnts, w, sw, out_dtype=torch.float32)
        want = ref.scaled_sums(a, sa, w[0], sw[0])
        assert torch.equal(torch.nan_to_num(out, nan=12345.0), torch.nan_to_num(want, nan=12345.0))
        assert torch.equal(out.isnan(), want.isnan())


def test_gemm_last_rows_of_memory():
    """Operands that end where their allocation ends, K not a multiple of a step."""
    for rows, N, K in ((1, 16, 16), (33, 48, 176), (290, 272, 1040)):
        offs, cnts, _ = buckets([rows])
        check(ints(rows, K, seed=1), scales(rows, seed=2), offs, cnts, ints(1, N, K, seed=3),
              scales(1, N, seed=4))


@pytest.mark.parametrize("T,E,k,N,K", [(128, 128, 8, 2816, 4096), (4093, 64, 6, 2048, 1408),
                                       (5, 1, 1, 4096, 7168), (1000, 1, 1, 4096, 4096)])
def test_gemm_at_work(T, E, k, N, K):
    """Sizes of this library's workloads, routed, with and without the dispatch copy."""
    g = torch.Generator(device=DEV).manual_seed(T)
    logits = torch.randn(T, E, generator=g, device=DEV)
    shape = moe.Shape(T, 128, E, k, 1, 1, torch.bfloat16)
    idx, _ = moe.route(logits, k)
    d = moe.alloc_dispatch(shape, DEV)
    moe.dispatch_index(idx, shape, d)
    a, sa = ints(T, K, seed=1), scales(T, seed=2)
    w, sw = ints(E, N, K, seed=3), scales(E, N, seed=4)
    token = d["row_token"]
    offs, cnts = d["expert_offsets"], d["expert_counts"]
    check(a, sa, offs, cnts, w, sw, index=token)
    check(a[token.long()], sa[token.long()], offs, cnts, w, sw)


# ----------------------------------------------------------------------- FFN

def ffn_case(T, H, E, k, I, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    logits = torch.randn(T, E, generator=g, device=DEV)
    shape = moe.Shape(T, H, E, k, 1, 1, torch.bfloat16)
    idx, gate = moe.route(logits, k)
    d = moe.alloc_dispatch(shape, DEV)
    moe.dispatch_index(idx, shape, d)
    x = torch.randn(T, H, generator=g, device=DEV) * torch.exp(torch.randn(T, 1, generator=g, device=DEV))
    x, sx = moe.quantize_int8(x)
    # g of the size that SiLU bends: a few units for a row of ordinary size
    wg, sg = moe.quantize_int8(torch.randn(E, 2 * I, H, generator=g, device=DEV) * H ** -0.5)
    wd, sd = moe.quantize_int8(torch.randn(E, H, I, generator=g, device=DEV) * I ** -0.5)
    return shape, d, idx, gate, x, sx, wg, sg, wd, sd


def check_ffn(out, d, x, sx, wg, sg, wd, sd):
    token = d["row_token"].long()
    for e, (o, n) in enumerate(zip(d["expert_offsets"].tolist(), d["expert_counts"].tolist())):
        if n == 0:
            continue
        t = token[o:o + n]
        want, bound = ref.swiglu(x[t], sx[t], wg[e], sg[e], wd[e], sd[e])
        err = (out[o:o + n].double() - want).abs() - bound
        assert float(err.max()) <= 0, f"expert {e}: {float(err.max())} over the bound"


FFN = [(3000, 512, 2, 1, 1040), (2500, 1040, 3, 2, 880), (1, 128, 4, 2, 64), (3, 144, 5, 3, 48), (17, 512, 8, 2, 208), (64, 272, 1, 1, 16),
       (40, 256, 64, 8, 1408), (130, 400, 4, 4, 272), (600, 512, 4, 2, 640), (900, 1024, 3, 2, 1040),
       (128, 4096, 16, 8, 1408)]


@pytest.mark.parametrize("T,H,E,k,I", FFN)
def test_swiglu(T, H, E, k, I):
    print(f"[swiglu int8] T={T} H={H} E={E} k={k} I={I}", flush=True)
    shape, d, _, _, x, sx, wg, sg, wd, sd = ffn_case(T, H, E, k, I)
    offs, cnts, token = d["expert_offsets"], d["expert_counts"], d["row_token"]
    out = moe.expert_swiglu_int8(x, sx, offs, cnts, shape, wg, sg, wd, sd, row_token=token)
    check_ffn(out, d, x, sx, wg, sg, wd, sd)
    rows = moe.expert_swiglu_int8(x[token.long()], sx[token.long()], offs, cnts, shape, wg, sg, wd, sd)
    assert torch.equal(rows, out)


@pytest.mark.parametrize("H,E,k,I", [(272, 1, 1, 16), (144, 1, 1, 2048), (256, 1, 1, 2064),
                                     (2064, 3, 2, 1408), (128, 40, 8, 400), (512, 2, 1, 272)])
def test_swiglu_few_rows(H, E, k, I):
    """A few rows by themselves and among many: the same bits, whoever makes the inner rows
    integers; a NaN and inner rows past the range of fp32 among them."""
    shape, d, idx, _, x, sx, wg, sg, wd, sd = ffn_case(40, H, E, k, I, seed=6)
    sx = sx.clone()
    sx[2], sx[3] = float("nan"), 1e30
    many = moe.expert_swiglu_int8(x, sx, d["expert_offsets"], d["expert_counts"], shape, wg, sg, wd, sd,
                                  row_token=d["row_token"])
    for T in {1, 2, 3, 4, 5, 7, 8, 9} if k == 1 else {1, 8 // k, 8 // k + 1}:
        print(f"[few rows] H={H} E={E} k={k} I={I} T={T}", flush=True)
        few = moe.Shape(T, H, E, k, 1, 1, torch.bfloat16)
        b = moe.alloc_dispatch(few, DEV)
        moe.dispatch_index(idx[:T].contiguous(), few, b)
        out = moe.expert_swiglu_int8(x[:T], sx[:T], b["expert_offsets"], b["expert_counts"], few, wg, sg,
                                     wd, sd, row_token=b["row_token"])
        got, want = out[b["pos"].flatten().long()], many[d["pos"][:T].flatten().long()]
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(), want.nan_to_num())
        if T <= 2:
            check_ffn(out, b, x, sx, wg, sg, wd, sd)


@pytest.mark.parametrize("T,H,I", [(1, 256, 128), (40, 256, 384), (40, 272, 144), (300, 512, 640)])
def test_swiglu_weights_off_a_line(T, H, I):
    """Weights that begin 16 bytes past a line give the bits of those that begin on one."""
    shape, d, _, _, x, sx, wg, sg, wd, sd = ffn_case(T, H, 4, 2, I, seed=7)
    off = lambda w: torch.cat([w.new_zeros(16), w.flatten()])[16:].view(w.shape)
    args = d["expert_offsets"], d["expert_counts"], shape
    want = moe.expert_swiglu_int8(x, sx, *args, wg, sg, wd, sd, row_token=d["row_token"])
    assert torch.equal(moe.expert_swiglu_int8(x, sx, *args, off(wg), sg, off(wd), sd,
                                              row_token=d["row_token"]), want)


def test_swiglu_large_gates():
    """Gates of hundreds, where SiLU is the gate or nothing, and of zeros."""
    shape, d, _, _, x, sx, wg, sg, wd, sd = ffn_case(50, 256, 3, 1, 128, seed=3)
    for f in (300.0, 0.0, 1e-30):
        out = moe.expert_swiglu_int8(x, sx * f, d["expert_offsets"], d["expert_counts"], shape, wg, sg,
                                     wd, sd, row_token=d["row_token"])
        check_ffn(out, d, x, sx * f, wg, sg, wd, sd)


def test_swiglu_nan_row_stays_alone():
    """A token whose scale is NaN gives NaN in its own rows only."""
    shape, d, idx, _, x, sx, wg, sg, wd, sd = ffn_case(300, 256, 3, 2, 128, seed=4)
    args = (d["expert_offsets"], d["expert_counts"], shape, wg, sg, wd, sd)
    want = moe.expert_swiglu_int8(x, sx, *args, row_token=d["row_token"])
    sx = sx.clone()
    sx[11] = float("nan")
    out = moe.expert_swiglu_int8(x, sx, *args, row_token=d["row_token"])
    mine = torch.zeros(600, dtype=torch.bool, device=DEV)
    mine[d["pos"][11].long()] = True
    assert out[mine].isnan().all() and torch.equal(out[~mine], want[~mine])


def test_swiglu_leaves_other_rows():
    """Rows in no bucket, and a workspace full of NaN before the call."""
    shape, d, _, _, x, sx, wg, sg, wd, sd = ffn_case(120, 256, 4, 1, 144, seed=5)
    offs, cnts = d["expert_offsets"], d["expert_counts"].clone()
    cnts[2] -= 5
    ws = torch.full((moe.expert_swiglu_int8_workspace_bytes(shape, 144),), 0xFF, dtype=torch.uint8,
                    device=DEV)
    out = torch.full((120, 256), 9.0, dtype=torch.bfloat16, device=DEV)
    moe.expert_swiglu_int8(x, sx, offs, cnts, shape, wg, sg, wd, sd, row_token=d["row_token"],
                           expert_out=out, workspace=ws)
    o, n = int(offs[2]), int(cnts[2])
    assert (out[o + n:o + n + 5] == 9).all()
    out[o + n:o + n + 5] = moe.expert_swiglu_int8(x, sx, offs, d["expert_counts"], shape, wg, sg, wd, sd,
                                                  row_token=d["row_token"])[o + n:o + n + 5]
    check_ffn(out, d, x, sx, wg, sg, wd, sd)


def test_swiglu_few_rows_in_buckets():
    """Buckets of a few rows: with gaps, out of order, past the rows, and none."""
    shape, d, _, _, x, sx, wg, sg, wd, sd = ffn_case(8, 272, 4, 1, 144, seed=5)
    for offs, cnts in (([5, 0, 3, 8], [3, 2, 1, 1]), ([-1, 2, 7, 0], [3, 4, 2, 0]), ([0, 0, 0, 0], [0, 0, 0, 0]),
                       ([0, 4, 2, 6], [1, 1, 1, 1]), ([0, 0, 0, 0], [0, 0, 9, 0]), ([4, 0, 0, 0], [-1, 0, 4, 0])):
        live = [(e, o, n) for e, (o, n) in enumerate(zip(offs, cnts)) if o >= 0 and n > 0 and o + n <= 8]
        ws = torch.full((moe.expert_swiglu_int8_workspace_bytes(shape, 144),), 0xFF, dtype=torch.uint8, device=DEV)
        out = torch.full((8, 272), 9.0, dtype=torch.bfloat16, device=DEV)
        moe.expert_swiglu_int8(x, sx, torch.tensor(offs, **I32), torch.tensor(cnts, **I32), shape, wg, sg, wd, sd,
                               expert_out=out, workspace=ws)
        rest = torch.ones(8, dtype=torch.bool, device=DEV)
        for e, o, n in live:
            rest[o:o + n] = False
            y, bound = ref.swiglu(x[o:o + n], sx[o:o + n], wg[e], sg[e], wd[e], sd[e])
            assert ((out[o:o + n].double() - y).abs() <= bound).all(), (offs, e)
        assert (out[rest] == 9).all(), offs


# ------------------------------------------------------------------- together

def block_buffers(T, H, E, k, I, seed):
    """A layer's inputs and every buffer of a step, as a serving program holds them."""
    shape, d, idx, gate, _, _, wg, sg, wd, sd = ffn_case(T, H, E, k, I, seed)
    g = torch.Generator(device=DEV).manual_seed(seed + 100)
    bf = dict(device=DEV, dtype=torch.bfloat16)
    return dict(
        shape=shape, d=d, wg=wg, sg=sg, wd=wd, sd=sd, idx=idx, gate=gate,
        x=torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16),
        r=torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16),
        norm=(1 + 0.1 * torch.randn(H, generator=g, device=DEV)).to(torch.bfloat16),
        router=torch.randn(E, H, generator=g, device=DEV) * H ** -0.5,
        total=torch.empty(T, H, **bf), y=torch.empty(T, H, **bf), eo=torch.empty(T * k, H, **bf),
        out=torch.empty(T, H, **bf), logits=torch.empty(T, E, device=DEV),
        q=torch.empty(T, H, device=DEV, dtype=torch.int8), s=torch.empty(T, device=DEV),
        ws=torch.empty(moe.expert_swiglu_int8_workspace_bytes(shape, I), device=DEV, dtype=torch.uint8))


def block_step(b):
    """Norm, router, index, experts on the tokens where they lie, combine."""
    shape, d = b["shape"], b["d"]
    moe.add_rms_norm(b["x"], b["norm"], 1e-6, residual=b["r"], total=b["total"], y=b["y"], q=b["q"],
                     scale=b["s"])
    torch.matmul(b["y"].float(), b["router"].t(), out=b["logits"])
    moe.route(b["logits"], shape.k, topk_idx=b["idx"], topk_w=b["gate"])
    moe.dispatch_index(b["idx"], shape, d)
    moe.expert_swiglu_int8(b["q"], b["s"], d["expert_offsets"], d["expert_counts"], shape, b["wg"],
                           b["sg"], b["wd"], b["sd"], row_token=d["row_token"], expert_out=b["eo"],
                           workspace=b["ws"])
    moe.combine(b["eo"], b["gate"], d["pos"], shape, y=b["out"])


def check_block(b):
    t, y = ref.norm(b["x"], b["norm"], 1e-6, b["r"])
    assert torch.equal(b["total"].double(), t)
    assert ((b["y"].double() - y).abs() <= ref.half_step(y, torch.bfloat16)).all()
    ref.check_int8_rows(b["q"], b["s"], y)
    check_ffn(b["eo"], b["d"], b["q"], b["s"], b["wg"], b["sg"], b["wd"], b["sd"])
    rows = b["eo"].double()[b["d"]["pos"].long()]
    want = (rows * b["gate"].double().unsqueeze(-1)).sum(1)
    size = (rows.abs() * b["gate"].double().unsqueeze(-1)).sum(1)
    k = rows.shape[1]
    bound = size * k * 2.0 ** -24 * 1.01 + (want.abs() + size * k * 2.0 ** -24) * 2.0 ** -8 + 2.0 ** -133
    assert ((b["out"].double() - want).abs() <= bound).all()


@pytest.mark.parametrize("T,H,E,k,I", [(1, 512, 16, 4, 208), (33, 512, 16, 4, 208), (700, 512, 8, 2, 256)])
def test_block(T, H, E, k, I):
    b = block_buffers(T, H, E, k, I, seed=6)
    block_step(b)
    check_block(b)


@pytest.mark.parametrize("T,H,E,k,I", [(2, 512, 16, 4, 208), (5, 512, 16, 4, 208), (700, 512, 8, 2, 256)])
def test_block_captured(T, H, E, k, I):
    """Replayed with new inputs and eager calls on other buffers in between."""
    b, other = block_buffers(T, H, E, k, I, seed=7), block_buffers(T, H, E, k, I, seed=8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block_step(b)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block_step(b)
    for rep in range(4):
        b["x"].copy_(torch.randn(T, H, device=DEV))
        for name in ("total", "y", "eo", "out", "q", "s"):
            b[name].view(torch.uint8).fill_(0x5A)
        graph.replay()
        block_step(other)
        torch.cuda.synchronize()
        check_block(b)
        replayed = b["out"].clone()
        block_step(b)
        assert torch.equal(b["out"], replayed), rep
    check_block(other)


def test_two_streams():
    """Calls on two streams at once, each with its own buffers."""
    bs = [block_buffers(300, 512, 8, 2, 256, seed=9), block_buffers(40, 512, 16, 4, 208, seed=10)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for b, st in zip(bs, streams):
            with torch.cuda.stream(st):
                block_step(b)
    torch.cuda.synchronize()
    for b in bs:
        check_block(b)
