"""The paged 8-bit KV cache on the GPU against its 64-bit plain forms (tests/paged_ref.py)."""
import numpy as np
import pytest
import torch

import paged_ref as ref
from quantized_attention_layer_gb300 import hfa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_attention_layer_gb300 import build
    build.build()


def make(nh, nkv, hd, ps, num, mx, window=0, scale=None, softcap=0.0, flags=0, theta=1e4, eps=1e-6, **kw):
    d = hfa.hfa_paged_desc(num_heads=nh, num_kv_heads=nkv, head_dim=hd, page_size=ps, num_pages=num,
                           max_pages=mx, window=window, eps=eps, rope_theta=theta,
                           attn_scale=scale if scale is not None else hd ** -0.5, softcap=softcap, flags=flags)
    return hfa.Paged(d, **kw)


class Pool:
    def __init__(self, arrays, table):
        self.k, self.ks, self.v, self.vs = ref.dev(*arrays)
        self.table = ref.dev(table)
        self.pages = hfa.Pages(self.k, self.ks, self.v, self.vs, self.table, table)

    def host(self):
        return [t.cpu().numpy() for t in (self.k, self.ks, self.v, self.vs)]


def draw_rows(rng, T, heads, hd, dtype):
    x = torch.from_numpy(rng.standard_normal((T, heads, hd)).astype(np.float32))
    return x.to(dtype)


def check_appended(before, after, rows, cu, start, table, ps, s_tol=ref.S_TOL):
    """Codes and scales of one matrix after an append, every untouched byte as it was."""
    codes0, scales0 = before
    codes1, scales1 = after
    real, sc = ref.append_pages(rows, cu, start, table, ps, codes0, scales0)
    assert np.all(np.abs(scales1 - sc) <= s_tol * sc), np.abs(scales1 - sc).max()
    left = np.isnan(real)
    assert np.array_equal(codes1[left], codes0[left])
    off = np.abs(codes1[~left] - real[~left])
    assert off.size == 0 or off.max() <= ref.C_TOL, off.max()


@pytest.mark.parametrize("hd,ps,nkv,G,kind,norm,factors,vnorm", [
    (64, 16, 2, 1, torch.bfloat16, False, False, False),
    (64, 128, 1, 8, torch.float32, True, False, False),
    (128, 16, 8, 4, torch.bfloat16, True, False, False),
    (128, 32, 3, 5, torch.float32, True, True, True),
    (128, 64, 2, 3, torch.bfloat16, True, False, True),
    (128, 128, 2, 2, torch.bfloat16, True, False, False),
    (256, 16, 1, 7, torch.bfloat16, False, True, False),
    (256, 32, 2, 2, torch.float32, True, False, False),
    (256, 64, 2, 1, torch.bfloat16, True, True, False),
    (256, 128, 1, 2, torch.float32, False, False, True)])
def test_append(hd, ps, nkv, G, kind, norm, factors, vnorm):
    rng = np.random.default_rng(hd + ps)
    nh = nkv * G
    ns = [1, 0, ps, 3 * ps + 5, 7, 2 * ps, 1]
    start = np.array([0, 9, ps - 1, 2 * ps, 5 * ps + ps - 3, ps // 2, 6 * ps - 1], dtype=np.int32)
    cu = ref.ragged(ns)
    mx = 8
    table, num = ref.make_table(rng, [-(-(s + n) // ps) for s, n in zip(start, ns)], mx)
    arrays = ref.make_pool(rng, num, nkv, ps, hd)
    pool = Pool(arrays, table)
    w = [torch.rand(hd) + 0.5 for _ in range(2)] if norm else [None, None]
    ff = (rng.random(hd // 2) * 7 + 1).astype(np.float32) if factors else None
    p = make(nh, nkv, hd, ps, num, mx, flags=hfa.HFA_F_V_UNIT_NORM if vnorm else 0,
             w_q=None if w[0] is None else w[0].cuda(), w_k=None if w[1] is None else w[1].cuda(),
             rope_factors=ff)
    T = int(cu[-1])
    # a packed projection output with 8 more values between its rows
    wide = torch.zeros((T, (nh + 2 * nkv) * hd + 8), dtype=kind)
    x = draw_rows(rng, T, nh + 2 * nkv, hd, kind)
    wide[:, :x[0].numel()] = x.reshape(T, -1)
    wide = wide.cuda()
    rows = wide.as_strided((T, nh + 2 * nkv, hd), (wide.stride(0), hd, 1))
    q, k, v = rows[:, :nh], rows[:, nh:nh + nkv], rows[:, nh + nkv:]
    q_out = torch.full((T + 1, nh, hd), 7.0, dtype=kind, device="cuda")
    cud, sd = ref.dev(cu, start)
    p.hfa_paged_append(cud, cu, sd, start, q, k, v, pool.pages, q_out[:T])
    p.hfa_paged_check_status()
    assert torch.all(q_out[T] == 7)  # the row behind the last sequence
    xf = x.double().numpy()
    pos = np.concatenate([np.arange(s, s + n) for s, n in zip(start, ns)])
    qn, kn, vn = xf[:, :nh], xf[:, nh:nh + nkv], xf[:, nh + nkv:]
    if norm:
        qn = ref.norm_rows(qn, w[0].double().numpy(), 1e-6)
        kn = ref.norm_rows(kn, w[1].double().numpy(), 1e-6)
    if vnorm:
        vn = ref.norm_rows(vn, None, 1e-6)
    want = ref.rotate_rows(qn, pos, 1e4, ff)
    tol = ref.Y_TOL * ref.pair_len(qn) + (ref.BF16 * np.abs(want) if kind == torch.bfloat16 else 0)
    assert np.all(np.abs(q_out[:T].double().cpu().numpy() - want) <= tol)
    after = pool.host()
    check_appended(arrays[:2], after[:2], ref.rotate_rows(kn, pos, 1e4, ff), cu, start, table, ps)
    check_appended(arrays[2:], after[2:], vn, cu, start, table, ps)
    # again: nothing grows, so nothing but the same bytes is written
    p.hfa_paged_append(cud, cu, sd, start, q, k, v, pool.pages, q_out[:T])
    for a, b in zip(after, pool.host()):
        assert np.array_equal(a, b)


def test_append_token_by_token_grows_the_scale():
    rng = np.random.default_rng(5)
    hd, ps, nkv = 64, 32, 2
    table, num = ref.make_table(rng, [2, 2], 2)
    pool = Pool(ref.make_pool(rng, num, nkv, ps, hd), table)
    p = make(2, nkv, hd, ps, num, 2)
    cu = ref.ragged([1, 1])
    cud = ref.dev(cu)
    for step in range(40):
        start = np.array([step, step + 3], dtype=np.int32)
        # magnitudes that rise and fall, so that some steps grow the scale and some do not
        x = draw_rows(rng, 2, 2 * nkv, hd, torch.float32) * float(1.3 ** (step % 7))
        before = pool.host()
        xd = x.cuda()
        p.hfa_paged_append(cud, cu, ref.dev(start), start, None, xd[:, :nkv], xd[:, nkv:], pool.pages)
        after = pool.host()
        xf = x.double().numpy()
        check_appended(before[:2], after[:2], ref.rotate_rows(xf[:, :nkv], start, 1e4, None), cu, start, table, ps)
        check_appended(before[2:], after[2:], xf[:, nkv:], cu, start, table, ps)
    p.hfa_paged_check_status()


def test_append_far_positions():
    # the angle of the last position there can be, and of factors below 1
    rng = np.random.default_rng(8)
    hd, ps = 128, 128
    mx = (1 << 24) // ps - 1
    table = np.full((1, mx), -1, dtype=np.int32)
    table[0, -1] = 1
    pool = Pool(ref.make_pool(rng, 2, 1, ps, hd), table)
    ff = np.full(hd // 2, 0.75, dtype=np.float32)
    p = make(1, 1, hd, ps, 2, mx, rope_factors=ff)
    start = np.array([mx * ps - 3], dtype=np.int32)
    cu = ref.ragged([3])
    x = draw_rows(rng, 3, 3, hd, torch.float32)
    xd = x.cuda()
    out = torch.empty((3, 1, hd), device="cuda")
    p.hfa_paged_append(ref.dev(cu), cu, ref.dev(start), start, xd[:, :1], xd[:, 1:2], xd[:, 2:], pool.pages, out)
    xf = x.double().numpy()[:, :1]
    want = ref.rotate_rows(xf, start[0] + np.arange(3), 1e4, ff)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= ref.Y_TOL * ref.pair_len(xf))


def test_append_non_finite_zero_and_tiny_values():
    hd, ps, nkv = 64, 16, 1
    rng = np.random.default_rng(3)
    table = np.arange(6, dtype=np.int32).reshape(6, 1)
    arrays = ref.make_pool(rng, 6, nkv, ps, hd)
    pool = Pool(arrays, table)
    p = make(1, nkv, hd, ps, 6, 1)
    ns = [4, 4, 2, 2, 1, 1]
    start = np.array([0, 3, 0, 0, 5, 0], dtype=np.int32)
    cu = ref.ragged(ns)
    k = draw_rows(rng, 14, nkv, hd, torch.float32) * 0  # position-free: rotation of zeros
    v = draw_rows(rng, 14, nkv, hd, torch.float32)
    v[1, 0, 3] = float("nan")
    v[2, 0, 4] = float("inf")
    v[3, 0, 5] = float("-inf")
    v[5, 0, 6] = float("nan")
    v[8:10] = 0           # a page of zeros
    v[10:12] *= 1e-41     # a scale below the smallest normal f32
    v[12] = float("nan")  # nothing finite behind 5 old rows: they stay
    v[13] = float("inf")  # nothing finite at all: zeros
    p.hfa_paged_append(ref.dev(cu), cu, ref.dev(start), start, None, k.cuda(), v.cuda(), pool.pages)
    p.hfa_paged_check_status()
    after = pool.host()
    vf = v.double().numpy()
    check_appended(arrays[2:], after[2:], vf, cu, start, table, ps)
    assert np.isfinite(after[3]).all()
    assert after[2][0, 0, 1, 3] == 0 and after[2][0, 0, 2, 4] == 127 and after[2][0, 0, 3, 5] == -127
    assert after[3][2, 0] == 0 and after[3][3, 0] == 0 and not after[2][2, 0, :2].any()
    assert after[3][4, 0] == arrays[3][4, 0] and np.array_equal(after[2][4, 0, :5], arrays[2][4, 0, :5])


def test_append_rotates_queries_in_place():
    rng = np.random.default_rng(4)
    table, num = ref.make_table(rng, [2], 2)
    pool = Pool(ref.make_pool(rng, num, 1, 16, 64), table)
    p = make(4, 1, 64, 16, num, 2)
    cu, start = ref.ragged([20]), np.array([2], dtype=np.int32)
    x = draw_rows(rng, 20, 6, 64, torch.bfloat16).cuda()
    q = x[:, :4].contiguous()
    apart = torch.empty_like(q)
    p.hfa_paged_append(ref.dev(cu), cu, ref.dev(start), start, q, x[:, 4:5], x[:, 5:], pool.pages, apart)
    p.hfa_paged_append(ref.dev(cu), cu, ref.dev(start), start, q, x[:, 4:5], x[:, 5:], pool.pages, q)
    assert torch.equal(apart, q)


@pytest.mark.parametrize("hd,ps,nkv", [(64, 16, 3), (128, 32, 2), (128, 128, 1), (256, 64, 2)])
def test_read(hd, ps, nkv):
    rng = np.random.default_rng(hd)
    start = np.array([0, 5, ps - 1, 0, 2 * ps], dtype=np.int32)
    count = np.array([3 * ps + 1, 0, 2, ps, 1], dtype=np.int32)
    table, num = ref.make_table(rng, [-(-(s + c) // ps) for s, c in zip(start, count)], 5)
    arrays = ref.make_pool(rng, num, nkv, ps, hd)
    pool = Pool(arrays, table)
    p = make(nkv, nkv, hd, ps, num, 5)
    cap = 4 * ps + 3
    kc = torch.full((5, nkv, cap, hd), 9.0, dtype=torch.bfloat16, device="cuda")
    vc = torch.full_like(kc, 9.0)
    p.hfa_paged_read(ref.dev(start), start, ref.dev(count), count, pool.pages, kc, vc)
    p.hfa_paged_check_status()
    for got, codes, scales in ((kc, arrays[0], arrays[1]), (vc, arrays[2], arrays[3])):
        want = torch.full((5, nkv, cap, hd), 9.0)
        for b in range(5):
            for t in range(start[b], start[b] + count[b]):
                pg = table[b, t // ps]
                want[b, :, t] = torch.from_numpy(codes[pg, :, t % ps].astype(np.float32) * scales[pg][:, None])
        assert torch.equal(got.cpu(), want.to(torch.bfloat16))


def run_attention(seed, nh, nkv, hd, ps, ns, lens, kind, window=0, softcap=0.0, scale=None, bidir=False, poison=True,
                  q_mul=1.0, repeat=1):
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, dtype=np.int32)
    cu = ref.ragged(ns)
    mx = max(1, -(-int(lens.max()) // ps)) + 1
    counts = [-(-int(n) // ps) for n in lens]
    table, num = ref.make_table(rng, counts, mx, fill=-5)
    arrays = ref.make_pool(rng, num, nkv, ps, hd)
    T = int(cu[-1])
    q = draw_rows(rng, T, nh + 1, hd, torch.float32) * q_mul
    q = q.to(kind).cuda()[:, :nh]  # rows a head apart
    o_ref, bound = ref.attend(q.double().cpu().numpy(), cu, lens, arrays, table, ps,
                              scale if scale is not None else hd ** -0.5, softcap, window, bidir)
    if poison:
        # pages behind every row's window, and what no visible position uses
        used = np.zeros(num, dtype=bool)
        for b, L in enumerate(lens):
            n = int(ns[b])
            lo = max(0, int(L) - n - window + 1) if window else 0
            for j in range(mx):
                if j * ps < L and (j + 1) * ps > lo and n:
                    used[table[b, j]] = True
                else:
                    table[b, j] = 10 ** 6 + j
        arrays[1][~used] = np.nan
        arrays[3][~used] = np.inf
    pool = Pool(arrays, table)
    p = make(nh, nkv, hd, ps, num, mx, window=window, softcap=softcap, scale=scale,
             flags=hfa.HFA_F_BLOCK_BIDIR if bidir else 0)
    ws = torch.zeros(p.hfa_paged_workspace_bytes(len(ns), T), dtype=torch.uint8, device="cuda")
    o = torch.full((T + 1, nh, hd), 3.0, dtype=kind, device="cuda")
    cud, ld = ref.dev(cu, lens)
    first = None
    for _ in range(repeat):
        o[:T] = float("nan")
        p.hfa_paged_attention(cud, cu, ld, lens, q, pool.pages, ws, o[:T])
        p.hfa_paged_check_status()
        if first is None:
            first = o.clone()
        assert torch.equal(first.view(torch.uint8), o.view(torch.uint8))
    assert torch.all(o[T] == 3)
    got = o[:T].double().cpu().numpy()
    if kind == torch.bfloat16:
        # o rounded once (2^-8 of it); rows served by bf16 tensor-core operands also round
        # each weight once (2^-8 of sum p |v|, of which `bound` holds a known share)
        big = bound / 2.0 ** -19  # >= sum p |v|
        bound = bound + ref.BF16 * np.abs(o_ref) + ref.BF16 * np.minimum(big, row_weight(arrays, bound, o_ref))
    assert not np.isnan(got).any()
    assert np.all(np.abs(got - o_ref) <= bound), np.max(np.abs(got - o_ref) - bound)
    return got


def row_weight(arrays, bound, o_ref):
    """sum p |v| is at most the largest |v|."""
    scales = arrays[3][np.isfinite(arrays[3])]
    return np.full_like(o_ref, 127 * float(scales.max()))


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("ps,nkv,G", [(16, 2, 1), (32, 1, 4), (64, 3, 5), (128, 1, 8), (16, 2, 7)])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_attention_single_tokens(hd, ps, nkv, G, kind):
    lens = [1, 0, ps - 1, ps, ps + 1, 129, 700]
    run_attention(hd + ps, nkv * G, nkv, hd, ps, [1] * len(lens), lens, kind, repeat=2)


@pytest.mark.parametrize("hd,ps,G,window,softcap", [(128, 16, 4, 33, 0.0), (256, 32, 2, 128, 0.0),
                                                    (64, 64, 8, 1, 0.0), (128, 64, 5, 0, 30.0),
                                                    (64, 128, 3, 1000, 20.0)])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_attention_single_tokens_window_and_softcap(hd, ps, G, window, softcap, kind):
    run_attention(hd, 2 * G, 2, hd, ps, [1, 1, 0, 1, 1], [500, 33, 77, 1, 2000], kind, window=window,
                  softcap=softcap, scale=0.3, repeat=2)


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("ps,nkv,G", [(16, 2, 1), (32, 1, 4), (64, 1, 3), (128, 1, 8)])
def test_attention_blocks(hd, ps, nkv, G):
    # one row, few rows, a tile's rows and more, empty sequences, rows before position 0
    ns = [1, 2, 0, 16, 33, 130, 5]
    lens = [300, 2, 40, 16, 500, 257, 3]
    run_attention(hd + ps, nkv * G, nkv, hd, ps, ns, lens, torch.bfloat16, repeat=2)


@pytest.mark.parametrize("hd,ps,G,window,softcap,bidir", [(128, 16, 4, 40, 0.0, False), (256, 32, 2, 100, 0.0, False),
                                                          (64, 64, 8, 7, 0.0, False), (128, 64, 5, 0, 30.0, False),
                                                          (128, 32, 2, 0, 0.0, True), (64, 128, 3, 500, 20.0, False),
                                                          (256, 128, 8, 0, 15.0, True)])
def test_attention_blocks_window_softcap_bidirectional(hd, ps, G, window, softcap, bidir):
    run_attention(hd, G, 1, hd, ps, [70, 3, 1, 140], [300, 600, 90, 140], torch.bfloat16, window=window,
                  softcap=softcap, scale=0.2, bidir=bidir, repeat=2)


@pytest.mark.parametrize("hd,ps,nkv,G,window,softcap,bidir", [
    (64, 16, 3, 4, 0, 0.0, False), (128, 32, 2, 4, 0, 0.0, False), (128, 16, 1, 2, 33, 0.0, False),
    (64, 128, 2, 3, 300, 20.0, False), (128, 64, 40, 4, 0, 0.0, True), (128, 128, 2, 1, 0, 30.0, False),
    (64, 32, 50, 4, 17, 0.0, False)])
def test_attention_blocks_of_one_row_tile(hd, ps, nkv, G, window, softcap, bidir):
    """Every sequence has at most 128 rows x heads, one of them just that many; few items that
    CTAs share, and more items than that."""
    ns = [128 // G, 16, 0, 9, 1, 30]
    lens = [700, 1300, 50, 9, 200, 28 if not bidir else 64]
    run_attention(hd + ps + G, nkv * G, nkv, hd, ps, ns, lens, torch.bfloat16, window=window, softcap=softcap,
                  scale=0.2, bidir=bidir, repeat=2)


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_attention_long_single_sequence(kind):
    run_attention(1, 8, 2, 128, 64, [1], [20000], kind, repeat=2)


def test_attention_few_rows_of_a_long_sequence():
    run_attention(2, 4, 1, 128, 32, [16], [9000], torch.bfloat16, repeat=2)


def test_attention_large_and_small_queries():
    # queries far from 1 (the kernels hold them in 16-bit parts)
    for mul in (1e-6, 3e4):
        run_attention(3, 4, 2, 64, 16, [1, 1], [90, 300], torch.float32, q_mul=mul, scale=0.02 / mul)
        run_attention(3, 4, 2, 64, 16, [1, 40], [90, 300], torch.bfloat16, q_mul=mul, scale=0.02 / mul)


def test_attention_pages_of_very_different_scales():
    rng = np.random.default_rng(0)
    for n, kind in ((1, torch.float32), (30, torch.bfloat16)):
        nh, nkv, hd, ps, L = 4, 1, 64, 16, 200
        table, num = ref.make_table(rng, [13], 13)
        arrays = ref.make_pool(rng, num, nkv, ps, hd)
        arrays[1][:] = 0.03 * 10.0 ** rng.uniform(-3, 0, arrays[1].shape)
        arrays[3][:] = 10.0 ** rng.uniform(-6, 3, arrays[3].shape)
        arrays[3][table[0, 2]] = 0
        arrays[1][table[0, 4]] = 0
        pool = Pool(arrays, table)
        p = make(nh, nkv, hd, ps, num, 13)
        cu, lens = ref.ragged([n]), np.array([L], dtype=np.int32)
        q = draw_rows(rng, n, nh, hd, kind).cuda()
        o = torch.empty_like(q)
        ws = torch.zeros(p.hfa_paged_workspace_bytes(1, n), dtype=torch.uint8, device="cuda")
        p.hfa_paged_attention(ref.dev(cu), cu, ref.dev(lens), lens, q, pool.pages, ws, o)
        want, bound = ref.attend(q.double().cpu().numpy(), cu, lens, arrays, table, ps, hd ** -0.5)
        if kind == torch.bfloat16:
            # weights and o rounded once each
            bound = bound + ref.BF16 * np.abs(want) + ref.BF16 * bound / 2.0 ** -19
        assert np.all(np.abs(o.double().cpu().numpy() - want) <= bound)


def serve(kind=torch.bfloat16, graph=False):
    """Prompts appended and attended in two chunks, then single tokens, against the oracle on
    the pool the appends left."""
    rng = np.random.default_rng(11)
    nh, nkv, hd, ps = 8, 2, 128, 16
    B, mx = 3, 12
    table, num = ref.make_table(rng, [12, 12, 12], mx)
    pool = Pool(ref.make_pool(rng, num, nkv, ps, hd), table)
    p = make(nh, nkv, hd, ps, num, mx, w_q=torch.rand(hd).cuda() + 0.5, w_k=torch.rand(hd).cuda() + 0.5)
    length = np.zeros(B, dtype=np.int32)
    for ns in ([40, 7, 0], [50, 0, 100], [1, 1, 1], [1, 1, 1], [1, 0, 1], [3, 1, 16]):
        cu = ref.ragged(ns)
        T = int(cu[-1])
        x = draw_rows(rng, T, nh + 2 * nkv, hd, kind).cuda()
        q = torch.empty((T, nh, hd), dtype=kind, device="cuda")
        o = torch.empty_like(q)
        start = length.copy()
        length = length + np.asarray(ns, dtype=np.int32)
        ws = torch.zeros(p.hfa_paged_workspace_bytes(B, T), dtype=torch.uint8, device="cuda")
        cud, sd, ld = ref.dev(cu, start, length)
        p.hfa_paged_append(cud, cu, sd, start, x[:, :nh], x[:, nh:nh + nkv], x[:, nh + nkv:], pool.pages, q)
        p.hfa_paged_attention(cud, cu, ld, length, q, pool.pages, ws, o)
        p.hfa_paged_check_status()
        want, bound = ref.attend(q.double().cpu().numpy(), cu, length, pool.host(), table, ps, hd ** -0.5)
        bound = bound + ref.BF16 * np.abs(want) + ref.BF16 * np.minimum(bound / 2.0 ** -19, 127 * float(pool.vs.max()))
        assert np.all(np.abs(o.double().cpu().numpy() - want) <= bound)
    return p, pool, table, length


def test_prompt_then_steps():
    serve()


def test_paged_prompt_to_linear_decode():
    """The pages of a served batch read into linear caches, and the linear attention on them:
    the joint path of hfa_paged_read and hfa_attention_decode."""
    p, pool, table, length = serve()
    nh, nkv, hd, ps = 8, 2, 128, 16
    C = 192
    kc = torch.zeros((3, nkv, C, hd), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    zero = np.zeros(3, dtype=np.int32)
    p.hfa_paged_read(ref.dev(zero), zero, ref.dev(length), length, pool.pages, kc, vc)
    q = torch.randn((3, nh, hd), device="cuda")
    desc = hfa.hfa_attn_desc(num_heads=nh, num_kv_heads=nkv, head_dim=hd, layer_type=1, window=0, kv_capacity=C,
                             attn_scale=hd ** -0.5, softcap=0.0, flags=0)
    pos = length - 1
    ws = torch.zeros(hfa.hfa_attention_workspace_bytes(desc, 3), dtype=torch.uint8, device="cuda")
    lin = hfa.hfa_attention_decode(desc, q, ref.dev(pos), pos, kc, vc, ws, torch.empty_like(q))
    cu = ref.ragged([1, 1, 1])
    ws2 = torch.zeros(p.hfa_paged_workspace_bytes(3, 3), dtype=torch.uint8, device="cuda")
    paged = p.hfa_paged_attention(ref.dev(cu), cu, ref.dev(length), length, q, pool.pages, ws2, torch.empty_like(q))
    # the linear cache holds each value rounded to bf16: logits off by 2^-8 of their absolute
    # sum, values by 2^-8 of theirs
    arrays = pool.host()
    _, bound = ref.attend(q.double().cpu().numpy(), cu, length, arrays, table, ps, hd ** -0.5)
    assert np.all(np.abs((lin - paged).double().cpu().numpy()) <= bound / 2.0 ** -19 * 2.0 ** -8 * 1.01 + 2 * bound)


@pytest.mark.parametrize("n", [1, 20])
def test_graph_replays_with_other_lengths(n):
    """Append and attention captured once, replayed at later positions on a side stream, two
    graphs with workspaces of their own in flight on two streams."""
    rng = np.random.default_rng(21)
    nh, nkv, hd, ps, mx, B = 4, 2, 64, 16, 20, 2
    p = make(nh, nkv, hd, ps, 2 * mx * B + 2, mx)
    cu = ref.ragged([n] * B)
    T = n * B
    sides = []
    for g in range(2):
        table, _ = ref.make_table(rng, [mx] * B, mx)
        arrays = ref.make_pool(rng, 2 * mx * B + 2, nkv, ps, hd)
        pool = Pool(arrays, table)
        start = np.array([200, 37], dtype=np.int32)
        x = draw_rows(rng, T, nh + 2 * nkv, hd, torch.bfloat16).cuda()
        s = dict(pool=pool, table=table, x=x, q=torch.empty((T, nh, hd), dtype=torch.bfloat16, device="cuda"),
                 o=torch.empty((T, nh, hd), dtype=torch.bfloat16, device="cuda"), cu=ref.dev(cu),
                 start=ref.dev(start), len=ref.dev(start + n), stream=torch.cuda.Stream(),
                 ws=torch.zeros(p.hfa_paged_workspace_bytes(B, T), dtype=torch.uint8, device="cuda"))

        def call(s=s, start=start, pool=pool):
            xx = s["x"]
            p.hfa_paged_append(s["cu"], cu, s["start"], start, xx[:, :nh], xx[:, nh:nh + nkv], xx[:, nh + nkv:],
                               pool.pages, s["q"])
            p.hfa_paged_attention(s["cu"], cu, s["len"], start + n, s["q"], pool.pages, s["ws"], s["o"])

        torch.cuda.synchronize()
        with torch.cuda.stream(s["stream"]):
            call()
        s["stream"].synchronize()
        s["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(s["graph"], stream=s["stream"]):
            call()
        sides.append(s)
    for start in ([0, 0], [5, 250], [299, 16]):
        start = np.array(start, dtype=np.int32)
        for s in sides:
            s["start"].copy_(ref.dev(start))
            s["len"].copy_(ref.dev(start + n))
        torch.cuda.synchronize()
        for s in sides:
            with torch.cuda.stream(s["stream"]):
                s["graph"].replay()
        torch.cuda.synchronize()
        p.hfa_paged_check_status()
        for s in sides:
            want, bound = ref.attend(s["q"].double().cpu().numpy(), cu, start + n, s["pool"].host(), s["table"], ps,
                                     hd ** -0.5)
            bound = bound + ref.BF16 * np.abs(want) + ref.BF16 * np.minimum(
                bound / 2.0 ** -19, 127 * float(s["pool"].vs.max()))
            assert np.all(np.abs(s["o"].double().cpu().numpy() - want) <= bound)


def test_pages_and_positions_found_wrong_on_the_device():
    """A replay may bring a table entry outside the pool or a length past the table: skipped,
    recorded, everything else served."""
    rng = np.random.default_rng(31)
    nh, nkv, hd, ps, mx = 4, 2, 64, 16, 4
    for n in (1, 20):
        table, num = ref.make_table(rng, [4, 4, 4], mx)
        arrays = ref.make_pool(rng, num, nkv, ps, hd)
        pool = Pool(arrays, table)
        p = make(nh, nkv, hd, ps, num, mx)
        bad = table.copy()
        bad[1, 3] = num
        bad[1, 1] = -1
        pool.table.copy_(ref.dev(bad))
        cu, lens = ref.ragged([n] * 3), np.array([60, 64, 30], dtype=np.int32)
        wrong = np.array([60, 64, 65], dtype=np.int32)
        q = draw_rows(rng, 3 * n, nh, hd, torch.bfloat16).cuda()
        o = torch.zeros_like(q)
        ws = torch.zeros(p.hfa_paged_workspace_bytes(3, 3 * n), dtype=torch.uint8, device="cuda")
        p.hfa_paged_attention(ref.dev(cu), cu, ref.dev(wrong), lens, q, pool.pages, ws, o)
        with pytest.raises(hfa.HfaError) as e:
            p.hfa_paged_check_status()
        assert e.value.status == hfa.HFA_EDEVICE
        p.hfa_paged_check_status()  # cleared
        want, bound = ref.attend(q.double().cpu().numpy(), cu, lens, arrays, table, ps, hd ** -0.5)
        bound = bound + ref.BF16 * np.abs(want) + ref.BF16 * bound / 2.0 ** -19
        got = o.double().cpu().numpy()
        assert np.all(np.abs(got - want)[:n] <= bound[:n])
        assert np.isfinite(got).all()
        # the append skips the same pages
        start = lens - n
        x = draw_rows(rng, 3 * n, nh + 2 * nkv, hd, torch.bfloat16).cuda()
        p.hfa_paged_append(ref.dev(cu), cu, ref.dev(start), start, x[:, :nh], x[:, nh:nh + nkv], x[:, nh + nkv:],
                           pool.pages, q)
        with pytest.raises(hfa.HfaError):
            p.hfa_paged_check_status()
        kc = torch.zeros((3, nkv, 64, hd), dtype=torch.bfloat16, device="cuda")
        zero = np.zeros(3, dtype=np.int32)
        p.hfa_paged_read(ref.dev(zero), zero, ref.dev(lens), lens, pool.pages, kc, torch.zeros_like(kc))
        with pytest.raises(hfa.HfaError):
            p.hfa_paged_check_status()


def test_pool_past_32_bit_offsets():
    """Pages whose codes lie beyond 4 GiB from the pool's start."""
    hd, ps, nkv, nh = 256, 128, 4, 4
    num = (1 << 32) // (hd * ps * nkv) + 40
    rng = np.random.default_rng(41)
    small = ref.make_pool(rng, 3, nkv, ps, hd)
    mx = 3
    table = np.array([[num - 1, num - 3, num - 7]], dtype=np.int32)
    k = torch.empty((num, nkv, ps, hd), dtype=torch.int8, device="cuda")
    v = torch.empty((num, nkv, ps, hd), dtype=torch.int8, device="cuda")
    ks = torch.full((num, nkv), float("nan"), device="cuda")
    vs = torch.full((num, nkv), float("nan"), device="cuda")
    at = torch.from_numpy(table[0].astype(np.int64)).cuda()
    for t, a in ((k, small[0]), (ks, small[1]), (v, small[2]), (vs, small[3])):
        t[at] = ref.dev(a)
    pages = hfa.Pages(k, ks, v, vs, ref.dev(table), table)
    p = make(nh, nkv, hd, ps, num, mx)
    for n, kind in ((1, torch.float32), (20, torch.bfloat16)):
        cu, lens = ref.ragged([n]), np.array([300], dtype=np.int32)
        q = draw_rows(rng, n, nh, hd, kind).cuda()
        o = torch.empty_like(q)
        ws = torch.zeros(p.hfa_paged_workspace_bytes(1, n), dtype=torch.uint8, device="cuda")
        p.hfa_paged_attention(ref.dev(cu), cu, ref.dev(lens), lens, q, pages, ws, o)
        want, bound = ref.attend(q.double().cpu().numpy(), cu, lens, small, np.array([[0, 1, 2]]), ps, hd ** -0.5)
        if kind == torch.bfloat16:
            bound = bound + ref.BF16 * np.abs(want) + ref.BF16 * bound / 2.0 ** -19
        assert np.all(np.abs(o.double().cpu().numpy() - want) <= bound)
    # append into the far pages, read back
    x = draw_rows(rng, 9, 2 * nkv, hd, torch.float32)
    cu, start = ref.ragged([9]), np.array([295], dtype=np.int32)
    xd = x.cuda()
    p.hfa_paged_append(ref.dev(cu), cu, ref.dev(start), start, None, xd[:, :nkv], xd[:, nkv:], pages)
    after = k[at].cpu().numpy(), ks[at].cpu().numpy()
    xf = x.double().numpy()
    check_appended(small[:2], after, ref.rotate_rows(xf[:, :nkv], 295 + np.arange(9), 1e4, None), cu, start,
                   np.array([[0, 1, 2]]), ps)
    kc = torch.zeros((1, nkv, 304, hd), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    count = np.array([9], dtype=np.int32)
    p.hfa_paged_read(ref.dev(start), start, ref.dev(count), count, pages, kc, vc)
    page = after[0][2].astype(np.float32) * after[1][2][:, None, None]
    assert torch.equal(kc[0, :, 295:].cpu(), torch.from_numpy(page[:, 39:48]).to(torch.bfloat16))
    p.hfa_paged_check_status()


def test_shared_prefix_pages():
    """Two sequences that read the same first pages."""
    rng = np.random.default_rng(51)
    nh, nkv, hd, ps = 4, 1, 128, 16
    table, num = ref.make_table(rng, [5, 5], 5)
    table[1, :3] = table[0, :3]
    arrays = ref.make_pool(rng, num, nkv, ps, hd)
    pool = Pool(arrays, table)
    p = make(nh, nkv, hd, ps, num, 5)
    for ns in ([1, 1], [12, 3]):
        cu, lens = ref.ragged(ns), np.array([70, 55], dtype=np.int32)
        q = draw_rows(rng, int(cu[-1]), nh, hd, torch.bfloat16).cuda()
        ws = torch.zeros(p.hfa_paged_workspace_bytes(2, int(cu[-1])), dtype=torch.uint8, device="cuda")
        o = p.hfa_paged_attention(ref.dev(cu), cu, ref.dev(lens), lens, q, pool.pages, ws, torch.empty_like(q))
        want, bound = ref.attend(q.double().cpu().numpy(), cu, lens, arrays, table, ps, hd ** -0.5)
        bound = bound + ref.BF16 * np.abs(want) + ref.BF16 * bound / 2.0 ** -19
        assert np.all(np.abs(o.double().cpu().numpy() - want) <= bound)


def test_refusals_with_a_handle():
    """Host checks of a live handle: nothing is launched, the message says what is wrong."""
    table = np.array([[0, 1, 2], [3, 4, 5]], dtype=np.int32)
    rng = np.random.default_rng(0)
    nh, nkv, hd, ps = 4, 2, 64, 16
    arrays = ref.make_pool(rng, 6, nkv, ps, hd)
    p = make(nh, nkv, hd, ps, 6, 3)
    x = torch.zeros((4, nh + 2 * nkv, hd), dtype=torch.bfloat16, device="cuda")
    q, k, v = x[:, :nh], x[:, nh:nh + nkv], x[:, nh + nkv:]
    out = torch.empty((4, nh, hd), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(p.hfa_paged_workspace_bytes(2, 4), dtype=torch.uint8, device="cuda")

    def status(call):
        with pytest.raises(hfa.HfaError) as e:
            call()
        assert str(e.value)
        return e.value.status

    def append(cu=(0, 2, 4), start=(0, 0), tab=table, q=q, k=k, v=v, out=out):
        pool = Pool(arrays, tab)
        cu, start = np.array(cu, dtype=np.int32), np.array(start, dtype=np.int32)
        p.hfa_paged_append(ref.dev(cu), cu, ref.dev(start), start, q, k, v, pool.pages, out)

    def attend(cu=(0, 2, 4), lens=(2, 2), q=q, out=out, ws=ws):
        pool = Pool(arrays, table)
        cu, lens = np.array(cu, dtype=np.int32), np.array(lens, dtype=np.int32)
        p.hfa_paged_attention(ref.dev(cu), cu, ref.dev(lens), lens, q, pool.pages, ws, out)

    assert status(lambda: append(cu=(1, 2, 4))) == hfa.HFA_EINVAL
    assert status(lambda: append(cu=(0, 5, 4))) == hfa.HFA_EINVAL
    assert status(lambda: append(start=(47, 0))) == hfa.HFA_ERANGE
    assert status(lambda: append(start=(-1, 0))) == hfa.HFA_ERANGE
    assert status(lambda: append(tab=np.array([[0, 1, 2], [0, 4, 5]], dtype=np.int32))) == hfa.HFA_EINVAL
    assert status(lambda: append(tab=np.array([[0, 1, 2], [6, 4, 5]], dtype=np.int32))) == hfa.HFA_EINVAL
    assert status(lambda: append(tab=np.array([[0, 1, 2], [-1, 4, 5]], dtype=np.int32))) == hfa.HFA_EINVAL
    # pages that the call does not write may be anything, also twice
    append(tab=np.array([[0, 9, 0], [5, 0, -3]], dtype=np.int32))
    append()  # the page check left nothing behind
    assert status(lambda: append(out=None)) == hfa.HFA_EINVAL
    assert status(lambda: append(k=k.float())) == hfa.HFA_EINVAL
    assert status(lambda: append(k=k[:3])) == hfa.HFA_EINVAL
    assert status(lambda: append(v=v.half())) == hfa.HFA_EINVAL
    odd = torch.zeros((4, nkv * hd + 4), dtype=torch.bfloat16, device="cuda")
    assert status(lambda: append(k=odd.as_strided((4, nkv, hd), (nkv * hd + 4, hd, 1)))) == hfa.HFA_EINVAL
    assert status(lambda: append(k=odd.view(-1)[4:4 + 4 * nkv * hd].view(4, nkv, hd))) == hfa.HFA_EINVAL
    assert status(lambda: attend(lens=(49, 2))) == hfa.HFA_ERANGE
    assert status(lambda: attend(lens=(-1, 2))) == hfa.HFA_ERANGE
    assert status(lambda: attend(q=q.half(), out=out.half())) == hfa.HFA_EINVAL
    assert status(lambda: attend(out=out.float())) == hfa.HFA_EINVAL
    assert status(lambda: attend(ws=ws[:16])) == hfa.HFA_EINVAL
    nine = torch.zeros((5, nh, hd), device="cuda")  # 5 rows of 2 heads: 10 rows at once
    assert status(lambda: attend(cu=(0, 5, 5), lens=(5, 0), q=nine, out=torch.empty_like(nine))) == hfa.HFA_EUNSUPPORTED
    cache = torch.zeros((2, nkv, 20, hd), dtype=torch.bfloat16, device="cuda")

    def read(start=(0, 0), count=(2, 2), cache=cache):
        pool = Pool(arrays, table)
        start, count = np.array(start, dtype=np.int32), np.array(count, dtype=np.int32)
        p.hfa_paged_read(ref.dev(start), start, ref.dev(count), count, pool.pages, cache, cache.clone())

    assert status(lambda: read(start=(19, 0))) == hfa.HFA_ERANGE
    assert status(lambda: read(count=(-1, 0))) == hfa.HFA_ERANGE
    assert status(lambda: read(cache=cache.float())) == hfa.HFA_EINVAL
    # nothing to do is not an error
    append(cu=(0, 0, 0), q=q[:0], k=k[:0], v=v[:0], out=out[:0])
    attend(cu=(0, 0, 0), lens=(5, 0), q=q[:0], out=out[:0])
    read(count=(0, 0))
    other = hfa.hfa_paged_desc.from_buffer_copy(p.desc)
    other.num_pages = 7
    p2 = hfa.Paged(other)
    pool = Pool(arrays, table)
    z = np.zeros(2, dtype=np.int32)
    assert status(lambda: p2.hfa_paged_read(ref.dev(z), z, ref.dev(z), z, pool.pages, cache, cache)) == hfa.HFA_EINVAL
    torch.cuda.synchronize()
    p.hfa_paged_check_status()


def test_one_workspace_for_calls_of_every_size():
    """A workspace as large as the largest call needs, used by calls of other batch sizes, row
    counts and handles in turn, eagerly and by two captured graphs: each finds it as a fresh one."""
    rng = np.random.default_rng(61)
    sides = []
    for nh, nkv, hd, ps, ns, lens in ((8, 2, 128, 16, [1], [3000]), (4, 4, 64, 32, [1] * 90, None),
                                      (8, 2, 128, 16, [20, 1], [900, 1200]), (2, 1, 256, 64, [2, 40, 1], [500, 700, 1])):
        lens = np.asarray(lens if lens is not None else rng.integers(1, 400, len(ns)), dtype=np.int32)
        mx = -(-int(lens.max()) // ps)
        table, num = ref.make_table(rng, [-(-int(n) // ps) for n in lens], mx)
        arrays = ref.make_pool(rng, num, nkv, ps, hd)
        cu = ref.ragged(ns)
        T = int(cu[-1])
        s = dict(p=make(nh, nkv, hd, ps, num, mx), pool=Pool(arrays, table), cu=cu, cud=ref.dev(cu), lens=lens,
                 ld=ref.dev(lens), q=draw_rows(rng, T, nh, hd, torch.bfloat16).cuda())
        s["o"] = torch.empty_like(s["q"])
        s["bytes"] = s["p"].hfa_paged_workspace_bytes(len(ns), T)
        s["want"], bound = ref.attend(s["q"].double().cpu().numpy(), cu, lens, arrays, table, ps, hd ** -0.5)
        s["bound"] = bound + ref.BF16 * np.abs(s["want"]) + ref.BF16 * bound / 2.0 ** -19
        sides.append(s)
    ws = torch.zeros(max(s["bytes"] for s in sides), dtype=torch.uint8, device="cuda")

    def call(s):
        s["p"].hfa_paged_attention(s["cud"], s["cu"], s["ld"], s["lens"], s["q"], s["pool"].pages, ws, s["o"])

    def check(s):
        s["p"].hfa_paged_check_status()
        assert np.all(np.abs(s["o"].double().cpu().numpy() - s["want"]) <= s["bound"])
        s["o"].fill_(float("nan"))

    for i in (0, 1, 2, 3, 1, 0, 2, 1, 3, 0):
        call(sides[i])
        check(sides[i])
    stream = torch.cuda.Stream()
    graphs = []
    torch.cuda.synchronize()
    for s in sides:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=stream):
            call(s)
    for i in (1, 0, 3, 1, 2, 0, 1):
        with torch.cuda.stream(stream):
            graphs[i].replay()
        stream.synchronize()
        check(sides[i])


def test_launches_that_overlap_wait_for_their_inputs():
    """Calls in a row on one stream, each reading what the kernel before wrote, that one being
    slow: another library's copy, an append, an attention, a read; eagerly, captured, and
    captured with the queries written on a second stream."""
    rng = np.random.default_rng(71)
    nh, nkv, hd, ps, mx = 8, 2, 128, 16, 8
    table, num = ref.make_table(rng, [mx], mx)
    p = make(nh, nkv, hd, ps, num, mx)
    x = draw_rows(rng, 100, nh + 2 * nkv, hd, torch.bfloat16).cuda()
    cu, start, lens = ref.ragged([100]), np.zeros(1, dtype=np.int32), np.array([100], dtype=np.int32)
    one, l1 = ref.ragged([1]), np.array([100], dtype=np.int32)
    cud, sd, ld, oned, l1d = ref.dev(cu, start, lens, one, l1)
    arrays = ref.make_pool(rng, num, nkv, ps, hd)
    ws = torch.zeros(p.hfa_paged_workspace_bytes(1, 100), dtype=torch.uint8, device="cuda")
    side, main = torch.cuda.Stream(), torch.cuda.Stream()

    def fresh():
        kc = torch.zeros((1, nkv, 128, hd), dtype=torch.bfloat16, device="cuda")
        o = torch.empty((100, nh, hd), dtype=torch.bfloat16, device="cuda")
        return dict(pool=Pool(arrays, table), x=torch.zeros_like(x), q=torch.zeros_like(o), o=o, o1=torch.zeros_like(o[:1]),
                    kc=kc, vc=torch.zeros_like(kc))

    def chain(s, forked, wait):
        def write():
            if wait:
                torch.cuda._sleep(2_000_000)
            s["x"].copy_(x)

        if forked:
            side.wait_stream(main)
            with torch.cuda.stream(side):
                write()
            main.wait_stream(side)
        else:
            write()
        y = s["x"]
        p.hfa_paged_append(cud, cu, sd, start, y[:, :nh], y[:, nh:nh + nkv], y[:, nh + nkv:], s["pool"].pages, s["q"])
        p.hfa_paged_attention(cud, cu, ld, lens, s["q"], s["pool"].pages, ws, s["o"])
        p.hfa_paged_attention(oned, one, l1d, l1, s["o"][99:], s["pool"].pages, ws, s["o1"])
        p.hfa_paged_read(sd, start, ld, lens, s["pool"].pages, s["kc"], s["vc"])

    def result(s):
        return [s[n].clone() for n in ("q", "o", "o1", "kc", "vc")] + [s["pool"].k.clone(), s["pool"].vs.clone()]

    # every kernel alone
    s = fresh()
    s["x"].copy_(x)
    torch.cuda.synchronize()
    p.hfa_paged_append(cud, cu, sd, start, x[:, :nh], x[:, nh:nh + nkv], x[:, nh + nkv:], s["pool"].pages, s["q"])
    torch.cuda.synchronize()
    p.hfa_paged_attention(cud, cu, ld, lens, s["q"], s["pool"].pages, ws, s["o"])
    torch.cuda.synchronize()
    p.hfa_paged_attention(oned, one, l1d, l1, s["o"][99:], s["pool"].pages, ws, s["o1"])
    torch.cuda.synchronize()
    p.hfa_paged_read(sd, start, ld, lens, s["pool"].pages, s["kc"], s["vc"])
    want = result(s)
    assert float(want[2].abs().max()) > 0
    for forked in (False, True):
        s = fresh()
        torch.cuda.synchronize()
        with torch.cuda.stream(main):
            chain(s, forked, True)
        main.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(result(s), want))
        s = fresh()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=main):
            chain(s, forked, True)
        for _ in range(3):
            for t in ("x", "q", "o", "o1", "kc", "vc"):
                s[t].zero_()
            torch.cuda.synchronize()
            with torch.cuda.stream(main):
                graph.replay()
            main.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(result(s), want))
    p.hfa_paged_check_status()


def test_refuses_tensors_off_the_device():
    table = np.array([[0, 1]], dtype=np.int32)
    arrays = ref.make_pool(np.random.default_rng(0), 2, 1, 16, 64)
    pool = Pool(arrays, table)
    with pytest.raises(hfa.HfaError) as e:
        hfa.Pages(pool.k.cpu(), pool.ks, pool.v, pool.vs, pool.table, table)
    assert e.value.status == hfa.HFA_EINVAL
    with pytest.raises(hfa.HfaError):
        hfa.Pages(pool.k, pool.ks, pool.v, pool.vs, pool.table.cpu(), table)
    with pytest.raises(hfa.HfaError):
        make(1, 1, 64, 16, 2, 2, w_q=torch.ones(64))
    p = make(1, 1, 64, 16, 2, 2)
    cu, z, ln = ref.ragged([1]), np.zeros(1, dtype=np.int32), np.ones(1, dtype=np.int32)
    cud, zd, ld = ref.dev(cu, z, ln)
    x = torch.zeros((1, 1, 64), device="cuda")
    cache = torch.zeros((1, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(p.hfa_paged_workspace_bytes(1, 1), dtype=torch.uint8, device="cuda")

    def off(call, args):
        """Every tensor argument in turn in host memory."""
        call(*args)
        for i, a in enumerate(args):
            if isinstance(a, torch.Tensor):
                with pytest.raises(hfa.HfaError) as e:
                    call(*args[:i], a.cpu(), *args[i + 1:])
                assert e.value.status == hfa.HFA_EINVAL

    off(p.hfa_paged_append, [cud, cu, zd, z, x, x.clone(), x.clone(), pool.pages, x.clone()])
    off(p.hfa_paged_attention, [cud, cu, ld, ln, x, pool.pages, ws, x.clone()])
    off(p.hfa_paged_read, [zd, z, ld, ln, pool.pages, cache, cache.clone()])
    p.hfa_paged_check_status()


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_the_largest_batch(hd):
    """4096 sequences, some without rows, some with none of their positions visible."""
    rng = np.random.default_rng(81)
    ns = [0 if b % 7 == 3 else 2 if b % 11 == 5 else 1 for b in range(4096)]
    lens = rng.integers(0, 48, 4096)
    lens[4095] = 700
    run_attention(81 + hd, 2, 1, hd, 16, ns, lens, torch.bfloat16)
    with pytest.raises(hfa.HfaError) as e:
        run_attention(81 + hd, 2, 1, hd, 16, ns + [1], list(lens) + [3], torch.bfloat16, poison=False)
    assert e.value.status == hfa.HFA_EINVAL


def test_the_largest_batch_appended_and_read():
    rng = np.random.default_rng(82)
    B, nkv, hd, ps, mx = 4096, 1, 64, 16, 3
    ns = np.array([0 if b % 5 == 2 else 1 + b % 3 for b in range(B)], dtype=np.int32)
    start = rng.integers(0, mx * ps - 3, B).astype(np.int32)
    cu = ref.ragged(ns)
    T = int(cu[-1])
    table, num = ref.make_table(rng, [mx] * B, mx)
    arrays = ref.make_pool(rng, num, nkv, ps, hd)
    pool = Pool(arrays, table)
    p = make(nkv, nkv, hd, ps, num, mx)
    x = draw_rows(rng, T, 2, hd, torch.float32)
    xd = x.cuda()
    p.hfa_paged_append(ref.dev(cu), cu, ref.dev(start), start, None, xd[:, :1], xd[:, 1:], pool.pages)
    p.hfa_paged_check_status()
    after = pool.host()
    pos = np.concatenate([start[b] + np.arange(ns[b]) for b in range(B)])
    xf = x.double().numpy()
    check_appended(arrays[:2], after[:2], ref.rotate_rows(xf[:, :1], pos, 1e4, None), cu, start, table, ps)
    check_appended(arrays[2:], after[2:], xf[:, 1:], cu, start, table, ps)
    kc = torch.zeros((B, nkv, mx * ps, hd), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    p.hfa_paged_read(ref.dev(start), start, ref.dev(ns), ns, pool.pages, kc, vc)
    p.hfa_paged_check_status()
    seq = np.repeat(np.arange(B), ns)
    pg = table[seq, pos // ps]
    for got, codes, scales in ((kc, after[0], after[1]), (vc, after[2], after[3])):
        want = torch.from_numpy(codes[pg, 0, pos % ps].astype(np.float32) * scales[pg, 0][:, None]).to(torch.bfloat16)
        assert torch.equal(got.cpu()[seq, 0, pos], want)
        assert int((got != 0).any(-1).sum()) <= T
