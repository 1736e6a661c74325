"""The 4-bit KV cache on the GPU against the 64-bit reference (tests/kv4_reference.py)."""
import numpy as np
import pytest
import torch

import synth
from oracle import sparda_oracle as O
from tests import kv4_reference as R
from tests.parity import to64

pytestmark = pytest.mark.gpu

W16 = 2.0 ** -11                  # an attention weight as an fp16 operand


@pytest.fixture(scope="module")
def sb(cuda_ok):
    from block_sparse_attention_forecast_gb300 import build
    build.build()
    import block_sparse_attention_forecast_gb300.binding as b
    b.sparda_device_error(clear=True)
    return b


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _kv(shape, seed):
    dims = (shape.max_batch, shape.n_groups, shape.max_ctx, 128)
    K = synth.normal_bf16(dims, seed, 1)
    K[..., 5] *= 6                                        # a strong channel and an offset, as keys have
    K = (K.float() + 0.5 * synth.normal_bf16((1, shape.n_groups, 1, 128), seed, 2).float()).to(torch.bfloat16)
    return K, synth.normal_bf16(dims, seed, 3)


def _filled(sb, shape, K, V, T_list):
    """A LayerKV4 whose memory held garbage (0xff: NaN scales) before the prompt was written."""
    layer = sb.LayerKV4.empty(shape)
    layer.kv.fill_(0xff)
    sb.sparda_kv4_quantize(shape, layer, K.cuda(), V.cuda(), _i32(T_list), len(T_list))
    return layer


def _read(sb, shape, layer, T_list, fill=7.0):
    k = torch.full((shape.max_batch, shape.n_groups, shape.max_ctx, 128), fill, dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, fill)
    sb.sparda_kv4_dequantize(shape, layer, _i32(T_list), len(T_list), k, v)
    torch.cuda.synchronize()
    assert sb.sparda_device_error(clear=True) == 0
    return k.cpu(), v.cpu()


def _v16(V):
    """The value rows as the attention reads them (fp16), float64."""
    return R.grid_values(V, key=False)


def _bf(x):
    return torch.from_numpy(x).to(torch.bfloat16)


# ------------------------------------------------------------------ quantize / dequantize
@pytest.mark.parametrize("T_list,G,ctx", [([1, 2, 31, 32, 33, 63, 64], 1, 64), ([65, 127, 128, 129, 200], 3, 256),
                                          ([1000, 1, 4096], 2, 4096)])
def test_prompt_values_exact(sb, T_list, G, ctx):
    shape = sb.Shape(n_groups=G, heads_per_group=3, max_ctx=ctx, max_batch=len(T_list) + 1)
    K, V = _kv(shape, 11)
    layer = _filled(sb, shape, K, V, T_list)
    k, v = _read(sb, shape, layer, T_list)
    kr, vr = R.grid_values(K, True), _v16(V)
    for b, T in enumerate(T_list):
        assert torch.equal(k[b, :, :T], _bf(kr[b, :, :T])), T
        assert torch.equal(v[b, :, :T], _bf(vr[b, :, :T])), T
        assert (k[b, :, T:] == 7).all() and (v[b, :, T:] == 7).all()
    assert (k[len(T_list):] == 7).all()
    assert (layer.kv[len(T_list):] == 0xff).all()         # the sequence behind the batch
    # the grid's own promise: within half a step, plus the roundings of z (2^-8 / 2^-11 of |z|) and
    # of the value (the same of |x|)
    for X, ref, r in ((K, kr, 2.0 ** -8), (V, vr, 2.0 ** -11)):
        x = to64(X).reshape(-1, 32)
        y = ref.reshape(-1, 32)
        lo, hi = x.min(1, keepdims=True), x.max(1, keepdims=True)
        s = (hi - lo) / 15 * (1 + r)
        bound = s / 2 + r * (np.abs(lo) + 16 * s) * 1.01 + 15 * r * s + r * np.abs(x).max(1, keepdims=True) + 1e-30
        assert (np.abs(x - y) <= bound).all()


def test_prompt_codes_at_borders(sb):
    """Codes halfway between two levels or beside it, over all scales: exact at every one."""
    T, G = 8192, 4
    shape = sb.Shape(n_groups=G, max_ctx=T, max_batch=1)
    gen = torch.Generator().manual_seed(17)
    groups = (1, G, T, 4)                                  # 32 channels each

    def draw(lo, hi):
        return lo + (hi - lo) * torch.rand(groups + (1,), generator=gen, dtype=torch.float64)

    def rows(kind, lo, hi):
        """kind: 0 halves of a step (ties), 1 whole numbers of any range, 2 normal with an offset, 3 halves
        of a step with a few last bits; scaled by 2^lo .. 2^hi."""
        noise = torch.randn(groups + (32,), generator=gen, dtype=torch.float64)
        whole = torch.randint(0, 31, groups + (32,), generator=gen).double() / 2
        whole[..., 0], whole[..., 1] = 0, 15                # the step is 1, and every half is a tie
        wide = torch.floor(whole * draw(0.2, 12))
        shift = torch.floor(draw(-24, 24))
        x = torch.stack([whole + shift, wide + shift, noise + shift * draw(0, 4), whole * (1 + noise * 2.0 ** -7) + shift])[kind]
        return (x * 2.0 ** torch.floor(draw(lo, hi))).reshape(1, G, T, 128).to(torch.bfloat16)

    for kind in range(4):
        for lo, hi in ((-3, 3), (-40, 40), (-135, 127)):
            K, V = rows(kind, lo, hi), rows(kind, max(lo, -28), min(hi, 12))
            layer = _filled(sb, shape, K, V, [T])
            k, v = _read(sb, shape, layer, [T])
            assert np.array_equal(to64(k), to64(_bf(R.grid_values(K, True))), equal_nan=True), (kind, lo, hi)
            assert np.array_equal(to64(v), to64(_bf(_v16(V))), equal_nan=True), (kind, lo, hi)


def test_prompt_special_groups(sb):
    shape = sb.Shape(n_groups=1, max_ctx=64, max_batch=1)
    K, V = _kv(shape, 12)
    rows = [torch.zeros(128), torch.full((128,), 3.0), torch.full((128,), -1e-30), torch.full((128,), 1e38),
            torch.cat([torch.full((32,), x) for x in (float("inf"), float("nan"), float("-inf"), 2.0)]),
            torch.linspace(-3e38, 3e38, 128), torch.linspace(-7e4, 7e4, 128), torch.linspace(100, 100.5, 128),
            torch.linspace(-1e-39, 1e-39, 128), torch.linspace(1e-6, 3e-6, 128), -torch.zeros(128)]
    for r, x in enumerate(rows):
        K[0, 0, r] = x.to(torch.bfloat16)
        V[0, 0, r] = x.to(torch.bfloat16)
    K[0, 0, 20, 7] = float("nan")
    V[0, 0, 21, 100] = float("inf")
    layer = _filled(sb, shape, K, V, [64])
    k, v = _read(sb, shape, layer, [64])
    assert np.array_equal(to64(k), to64(_bf(R.grid_values(K, True))), equal_nan=True)
    assert np.array_equal(to64(v), to64(_bf(_v16(V))), equal_nan=True)
    assert torch.isnan(k[0, 0, 20, :32]).all() and not torch.isnan(k[0, 0, 20, 32:]).any()
    assert torch.isnan(k[0, 0, 4, :96]).all() and (k[0, 0, 4, 96:] == 2).all()


def test_dequantize_selected_blocks(sb):
    T_list = [300, 64, 700]
    shape = sb.Shape(n_groups=2, max_ctx=704, max_batch=4, topk=3)
    K, V = _kv(shape, 13)
    layer = _filled(sb, shape, K, V, T_list)
    full_k, full_v = _read(sb, shape, layer, T_list)
    idx = _i32([[[0, 4, 2, -1, -1], [4, 0, 0, 1, 3]], [[0, -1, -1, -1, -1]] * 2, [[10, 5, 3, 1, 0], [7, 9, -1, -1, -1]]])
    cnt = _i32([[3, 5], [1, 0], [5, 2]])
    st = torch.full((4, 2, 5, 64, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    sv = st.clone()
    sb.sparda_kv4_dequantize(shape, layer, _i32(T_list), 3, st, sv, idx=idx, cnt=cnt)
    torch.cuda.synchronize()
    assert sb.sparda_device_error(clear=True) == 0
    for b, T in enumerate(T_list):
        for g in range(2):
            for s in range(5):
                j = int(idx[b, g, s])
                live = max(0, min(64, T - 64 * j)) if s < int(cnt[b, g]) else 0
                assert torch.equal(st[b, g, s, :live].cpu(), full_k[b, g, 64 * j:64 * j + live])
                assert torch.equal(sv[b, g, s, :live].cpu(), full_v[b, g, 64 * j:64 * j + live])
                assert (st[b, g, s, live:] == 9).all() and (sv[b, g, s, live:] == 9).all()
    assert (st[3] == 9).all()
    # an index outside the sequence: reported, its slot left
    bad = idx.clone()
    bad[1, 0, 0] = 1
    st.fill_(9)
    sb.sparda_kv4_dequantize(shape, layer, _i32(T_list), 3, st, sv, idx=bad, cnt=cnt)
    torch.cuda.synchronize()
    assert sb.sparda_device_error(clear=True) == sb.DEV_BAD_INDEX
    assert (st[1, 0] == 9).all() and torch.equal(st[0, 0, 1, :44].cpu(), full_k[0, 0, 256:300])


# ------------------------------------------------------------------ append
def test_append_equals_prompt_token_by_token(sb):
    """From an empty cache of garbage, 150 tokens one at a time: the stored bytes of the values are
    those of a prompt, and every completed window's compressed key is the exact mean of its stored
    keys rounded to bf16."""
    n = 150
    shape = sb.Shape(n_groups=3, heads_per_group=1, max_ctx=192, max_batch=3)
    K, V = _kv(shape, 21)
    layer = sb.LayerKV4.empty(shape)
    layer.kv.fill_(0xff)
    layer.ck.fill_(5)
    seq = _i32([0, 30])                                        # the second sequence starts behind 30 tokens
    pre = _filled(sb, shape, K, V, [1, 30])
    layer.kv[1] = pre.kv[1]
    for step in range(n):
        seq += 1
        T = seq.tolist()
        kn = torch.stack([K[b, :, T[b] - 1] for b in range(2)]).cuda()
        vn = torch.stack([V[b, :, T[b] - 1] for b in range(2)]).cuda()
        sb.sparda_kv4_append(shape, layer, kn, vn, seq, 2)
        if step in (0, 1, 31, 63, 64, 65, n - 1):
            k, v = _read(sb, shape, layer, T)
            for b in range(2):
                assert torch.equal(k[b, :, :T[b]], _bf(R.grid_values(K[b, :, :T[b]], True))), (step, b)
                assert torch.equal(v[b, :, :T[b]], _bf(_v16(V[b, :, :T[b]]))), (step, b)
    kr = R.grid_values(K, True)
    for b in range(2):
        W = O.num_windows(T[b])
        for g in range(3):
            want = O.compress_keys(kr[b, g, :T[b]], W)
            # the second sequence's first 30 tokens came as a prompt, which leaves ck alone; every
            # window completes by a later append, so all are written
            assert np.array_equal(to64(layer.ck[b, g, :W]), want), (b, g)
    assert (layer.ck[:2, :, O.num_windows(180):] == 5).all() and (layer.ck[2] == 5).all()
    assert (layer.kv[2] == 0xff).all()


def test_append_reports_bad_lengths(sb):
    shape = sb.Shape(n_groups=1, max_ctx=128, max_batch=3)
    layer = sb.LayerKV4.empty(shape)
    layer.kv.fill_(0xaa)
    x = torch.ones((3, 1, 128), dtype=torch.bfloat16, device="cuda")
    sb.sparda_kv4_append(shape, layer, x, x, _i32([0, 129, -5]), 3)
    torch.cuda.synchronize()
    assert sb.sparda_device_error(clear=True) == sb.DEV_BAD_SEQ_LEN
    assert (layer.kv == 0xaa).all()


# ------------------------------------------------------------------ attention
def _check_attention(sb, shape, layer, K, V, T_list, q, idx, cnt, mass=False, ws=None):
    B, G, H = len(T_list), shape.n_groups, shape.heads_per_group
    out = torch.full((shape.max_batch, G * H, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    ws = ws if ws is not None else sb.workspace(shape, B, sb.WS_KV4_ATTN_MASS if mass else sb.WS_KV4_ATTN)
    m0 = m = None
    if mass:
        m = synth.normal_bf16((shape.max_batch, G, shape.max_ctx // 64), 99).float().abs().cuda()
        m0 = to64(m)
    sb.sparda_kv4_decode_attn(shape, layer, q.cuda(), idx, cnt, _i32(T_list), B, out, ws, mass=m)
    torch.cuda.synchronize()
    assert sb.sparda_device_error(clear=True) == 0
    assert (out[B:] == 3).all()
    o = to64(out)
    for b, T in enumerate(T_list):
        nb = (T - 1) // 64 + 1
        for g in range(G):
            blocks = None if idx is None else [int(x) for x in idx[b, g, :int(cnt[b, g])]]
            k = R.grid_values(K[b, g, :64 * nb], True)
            v = _v16(V[b, g, :64 * nb])
            ref, tol, w, wtol = R.attention(to64(q[b, g * H:(g + 1) * H]), k, v, blocks, T, W16)
            err = np.abs(o[b, g * H:(g + 1) * H] - ref)
            assert (err <= tol).all(), (b, g, T, float((err - tol).max()))
            if mass:
                want = m0[b, g].copy()
                per = np.zeros(shape.max_ctx // 64)
                for j, x in zip(blocks if blocks is not None else range(nb), w):
                    per[j] += x
                want += per
                err = np.abs(to64(m[b, g]) - want)
                assert (err <= wtol * per + 2.0 ** -22 * np.abs(want)).all(), (b, g, float(err.max()))
    if mass:
        assert np.array_equal(to64(m[B:]), m0[B:])
    return out


def _select(rng, T_list, G, topk):
    """Block 0, the tail block and up to topk others, ascending, -1 padded."""
    idx = -np.ones((len(T_list), G, topk + 2), dtype=np.int32)
    cnt = np.zeros((len(T_list), G), dtype=np.int32)
    for b, T in enumerate(T_list):
        tb = (T - 1) // 64
        for g in range(G):
            pool = np.arange(1, tb)
            pick = rng.choice(pool, size=min(topk, len(pool)), replace=False) if len(pool) else []
            sel = sorted({0, tb} | set(int(x) for x in pick))
            idx[b, g, :len(sel)] = sel
            cnt[b, g] = len(sel)
    return torch.from_numpy(idx).cuda(), torch.from_numpy(cnt).cuda()


CASES = [
    # T_list, G, H, ctx, topk (0: all blocks)
    ([1], 1, 1, 64, 0),
    ([1, 2, 15, 16, 17, 63, 64, 65], 2, 16, 128, 0),
    ([64, 128, 129, 1000], 3, 5, 1024, 0),
    ([5000], 2, 16, 5056, 0),
    ([33, 4097, 700], 1, 9, 4160, 0),
    ([1, 64, 65, 130], 2, 16, 192, 8),
    ([4096, 3000, 2500], 2, 16, 4096, 8),
    ([4096], 1, 8, 4096, 62),
    ([777] * 20, 2, 2, 832, 4),
    ([640, 100] * 40, 2, 4, 640, 0),
]


@pytest.mark.parametrize("mass", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(sb, case, mass):
    T_list, G, H, ctx, topk = CASES[case]
    B = len(T_list)
    shape = sb.Shape(n_groups=G, heads_per_group=H, max_ctx=ctx, max_batch=B + 1, topk=max(1, topk))
    K, V = _kv(shape, 31 + case)
    layer = _filled(sb, shape, K, V, T_list)
    q = synth.normal_bf16((B, G * H, 128), 32, case)
    idx, cnt = _select(np.random.default_rng(case), T_list, G, topk) if topk else (None, None)
    _check_attention(sb, shape, layer, K, V, T_list, q, idx, cnt, mass)


def test_attention_peaked_and_flat(sb):
    """Scores of a few units around and, scaled up, hundreds apart (the running maximum moves often
    and most weights vanish); and equal scores."""
    T_list = [3000]
    shape = sb.Shape(n_groups=1, heads_per_group=16, max_ctx=3008, max_batch=1)
    K, V = _kv(shape, 41)
    layer = _filled(sb, shape, K, V, T_list)
    q = synth.normal_bf16((1, 16, 128), 42)
    q[0, 4:8] = 0                                              # flat
    q[0, 8:] = (q[0, 8:].float() * 60).to(torch.bfloat16)      # peaked
    _check_attention(sb, shape, layer, K, V, T_list, q, None, None, mass=True)


def test_attention_selection_edges(sb):
    """cnt 0, a block named twice, unsorted blocks, cnt above topk+2 (clamped)."""
    T_list = [500, 500, 500, 500]
    shape = sb.Shape(n_groups=1, heads_per_group=4, max_ctx=512, max_batch=4, topk=2)
    K, V = _kv(shape, 51)
    layer = _filled(sb, shape, K, V, T_list)
    q = synth.normal_bf16((4, 4, 128), 52)
    idx = _i32([[[3, 3, 0, -1]], [[7, 0, 5, 2]], [[1, -1, -1, -1]], [[0, 1, 2, 7]]])
    cnt = _i32([[3], [4], [0], [4]])
    _check_attention(sb, shape, layer, K, V, T_list, q, idx, cnt, mass=True)
    out = torch.ones((4, 4, 128), dtype=torch.bfloat16, device="cuda")
    ws = sb.workspace(shape, 4, sb.WS_KV4_ATTN)
    sb.sparda_kv4_decode_attn(shape, layer, q.cuda(), idx, cnt, _i32(T_list), 4, out, ws)
    ref = out.clone()
    assert (out[2] == 0).all()
    over = cnt.clone()
    over[3] = 9
    sb.sparda_kv4_decode_attn(shape, layer, q.cuda(), idx, over, _i32(T_list), 4, out, ws)
    assert torch.equal(out, ref)
    # an index outside the sequence is reported and skipped: sequence 1 without its block 5
    bad, less = idx.clone(), idx.clone()
    bad[1, 0, 2] = 8
    less[1, 0] = torch.tensor([7, 0, 2, -1], dtype=torch.int32)
    c3 = cnt.clone()
    c3[1] = 3
    mass = torch.zeros((4, 1, 8), device="cuda")
    wm = sb.workspace(shape, 4, sb.WS_KV4_ATTN_MASS)
    sb.sparda_kv4_decode_attn(shape, layer, q.cuda(), bad, cnt, _i32(T_list), 4, out, wm, mass=mass)
    torch.cuda.synchronize()
    assert sb.sparda_device_error(clear=True) == sb.DEV_BAD_INDEX
    sb.sparda_kv4_decode_attn(shape, layer, q.cuda(), less, c3, _i32(T_list), 4, ref, ws)
    assert (out.float() - ref.float()).abs().max() <= 2.0 ** -7 * ref.float().abs().max()
    assert abs(float(mass[1].sum()) - 4) < 1e-3                # four heads, one each
    # lengths out of range: zero output, reported; the others are unaffected
    sb.sparda_kv4_decode_attn(shape, layer, q.cuda(), idx, cnt, _i32([500, 0, 500, 513]), 4, out, ws)
    torch.cuda.synchronize()
    assert sb.sparda_device_error(clear=True) == sb.DEV_BAD_SEQ_LEN
    assert (out[1] == 0).all() and (out[3] == 0).all()
    assert (out[0] != 0).any()


def test_attention_nan_rows(sb):
    """A NaN key group reaches only its own group's heads; masked garbage reaches nothing."""
    T_list = [100]
    shape = sb.Shape(n_groups=2, heads_per_group=2, max_ctx=128, max_batch=1)
    K, V = _kv(shape, 61)
    K[0, 1, 50, 3] = float("nan")
    layer = _filled(sb, shape, K, V, T_list)
    q = synth.normal_bf16((1, 4, 128), 62).cuda()
    out = torch.zeros((1, 4, 128), dtype=torch.bfloat16, device="cuda")
    sb.sparda_kv4_decode_attn(shape, layer, q, None, None, _i32(T_list), 1, out, sb.workspace(shape, 1, sb.WS_KV4_ATTN))
    assert not torch.isnan(out[0, :2]).any() and torch.isnan(out[0, 2:]).all()


def test_attention_many_groups(sb):
    """More (sequence, group)s than the balanced plan holds: whole groups per CTA."""
    B = 530
    T_list = [1 + (37 * b) % 190 for b in range(B)]
    shape = sb.Shape(n_groups=2, heads_per_group=2, max_ctx=192, max_batch=B, topk=1)
    K, V = _kv(shape, 71)
    layer = _filled(sb, shape, K, V, T_list)
    q = synth.normal_bf16((B, 4, 128), 72)
    _check_attention(sb, shape, layer, K, V, T_list, q, None, None, mass=True)
    idx, cnt = _select(np.random.default_rng(7), T_list, 2, 1)
    _check_attention(sb, shape, layer, K, V, T_list, q, idx, cnt)


def test_attention_offsets_past_32_bits(sb):
    """The last sequence of a cache of 5.4 GB, read and written beyond byte 2^32."""
    B, ctx = 64, 262144
    shape = sb.Shape(n_groups=2, heads_per_group=16, max_ctx=ctx, max_batch=B)
    layer = sb.LayerKV4.empty(shape)
    assert layer.kv.numel() > 1 << 32
    T_list = [70] * (B - 1) + [2000]
    K = torch.zeros((B, 2, ctx, 128), dtype=torch.bfloat16, device="cuda")
    V = torch.zeros_like(K)
    Ks, Vs = synth.normal_bf16((2, 2048, 128), 81, 1), synth.normal_bf16((2, 2048, 128), 81, 2)
    K[-1, :, :2048], V[-1, :, :2048] = Ks.cuda(), Vs.cuda()
    sb.sparda_kv4_quantize(shape, layer, K, V, _i32(T_list), B)
    q = synth.normal_bf16((B, 32, 128), 82)
    out = torch.zeros((B, 32, 128), dtype=torch.bfloat16, device="cuda")
    sb.sparda_kv4_decode_attn(shape, layer, q.cuda(), None, None, _i32(T_list), B, out, sb.workspace(shape, B, sb.WS_KV4_ATTN))
    torch.cuda.synchronize()
    assert sb.sparda_device_error(clear=True) == 0
    for g in range(2):
        ref, tol, _, _ = R.attention(to64(q[-1, 16 * g:16 * g + 16]), R.grid_values(Ks[g], True), _v16(Vs[g]), None, 2000, W16)
        assert (np.abs(to64(out[-1, 16 * g:16 * g + 16]) - ref) <= tol).all()


def test_attention_repeats_and_leaves_the_workspace(sb):
    """Calls back to back on one workspace, in a graph and on a side stream give the same bits."""
    T_list = [9000, 77, 5000]
    shape = sb.Shape(n_groups=2, heads_per_group=8, max_ctx=9024, max_batch=3)
    K, V = _kv(shape, 91)
    layer = _filled(sb, shape, K, V, T_list)
    q = synth.normal_bf16((3, 16, 128), 92).cuda()
    seq = _i32(T_list)
    ws = sb.workspace(shape, 3, sb.WS_KV4_ATTN_MASS)
    outs, masses = [], []
    for _ in range(3):
        outs.append(torch.zeros((3, 16, 128), dtype=torch.bfloat16, device="cuda"))
        masses.append(torch.zeros((3, 2, 141), device="cuda"))
        sb.sparda_kv4_decode_attn(shape, layer, q, None, None, seq, 3, outs[-1], ws, mass=masses[-1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o2, m2 = torch.zeros_like(outs[0]), torch.zeros_like(masses[0])
    side.wait_stream(torch.cuda.current_stream())
    sb.sparda_kv4_decode_attn(shape, layer, q, None, None, seq, 3, o2, ws, mass=m2, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    o3, m3 = torch.zeros_like(outs[0]), torch.zeros_like(masses[0])
    with torch.cuda.graph(graph):
        sb.sparda_kv4_decode_attn(shape, layer, q, None, None, seq, 3, o3, ws, mass=m3)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for o, m in zip(outs[1:] + [o2], masses[1:] + [m2]):
        # which CTA joins a group's partial results may differ, their order does not
        assert torch.equal(o, outs[0]) and torch.equal(m, masses[0])
    assert torch.equal(o3, outs[0])
    assert (m3 - 2 * masses[0]).abs().max() <= 2.0 ** -22 * m3.max()
    counters = ws[:3 * 2 * 4].view(torch.int32)
    assert (counters == 0).all()
    assert sb.sparda_device_error(clear=True) == 0


# ------------------------------------------------------------------ mass of the bf16 cache
@pytest.mark.parametrize("T_list,topk", [([4096, 3000, 65, 1], 8), ([2500] * 20, 8), ([4000], 62), ([300] * 90, 2)])
def test_bf16_attention_with_mass(sb, T_list, topk):
    B, G, ctx = len(T_list), 2, 4096
    shape = sb.Shape(n_groups=G, max_ctx=ctx, max_batch=B, topk=topk)
    layer = sb.LayerKV.empty(shape)
    K, V = synth.normal_bf16((B, G, ctx, 128), 101, 1), synth.normal_bf16((B, G, ctx, 128), 101, 2)
    layer.k.copy_(K.cuda())
    layer.v.copy_(V.cuda())
    q = synth.normal_bf16((B, 32, 128), 102)
    idx, cnt = _select(np.random.default_rng(3), T_list, G, topk)
    out, plain = (torch.zeros((B, 32, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    mass = torch.zeros((B, G, ctx // 64), device="cuda")
    ws = sb.workspace(shape, B, sb.WS_ATTN_MASS)
    sb.sparda_sparse_decode_attn(shape, layer, q.cuda(), idx, cnt, _i32(T_list), B, plain, ws)
    sb.sparda_sparse_decode_attn_mass(shape, layer, q.cuda(), idx, cnt, _i32(T_list), B, out, ws, mass)
    torch.cuda.synchronize()
    assert sb.sparda_device_error(clear=True) == 0
    assert torch.equal(out, plain)
    for b in range(0, B, max(1, B // 5)):
        for g in range(G):
            blocks = [int(x) for x in idx[b, g, :int(cnt[b, g])]]
            _, _, w, wtol = R.attention(to64(q[b, 16 * g:16 * g + 16]), to64(K[b, g]), to64(V[b, g]), blocks, T_list[b], 0)
            want = np.zeros(ctx // 64)
            want[blocks] = w
            got = to64(mass[b, g])
            assert (np.abs(got - want) <= (wtol + 2.0 ** -22) * want).all()
            assert abs(got.sum() - 16) < 1e-3


# ------------------------------------------------------------------ many blocks
@pytest.mark.parametrize("T_list,G,H,ctx", [
    ([16384, 1, 64, 65, 8191, 4000, 127, 12345], 2, 16, 16384),
    ([16320] * 5, 3, 3, 16384),
    ([1 + (53 * b) % 512 for b in range(400)], 2, 8, 512),       # several short groups per CTA
    ([70000], 4, 11, 70016),
])
def test_attention_many_blocks(sb, T_list, G, H, ctx):
    B = len(T_list)
    shape = sb.Shape(n_groups=G, heads_per_group=H, max_ctx=ctx, max_batch=B + 1)
    K, V = _kv(shape, 110 + B)
    layer = _filled(sb, shape, K, V, T_list)
    q = synth.normal_bf16((B, G * H, 128), 111, B)
    q[:, 0] = (q[:, 0].float() * 40).to(torch.bfloat16)          # peaked: the references move
    q[:, 1] = 0
    _check_attention(sb, shape, layer, K, V, T_list, q, None, None)


def test_attention_many_selected_blocks(sb):
    """Selections of up to 64 blocks in a large batch; empty ones, bad lengths and indices among them."""
    B, G, ctx, topk = 70, 1, 4096, 62
    T_list = [1 + (977 * b) % 4096 for b in range(B)]
    shape = sb.Shape(n_groups=G, heads_per_group=16, max_ctx=ctx, max_batch=B, topk=topk)
    K, V = _kv(shape, 121)
    layer = _filled(sb, shape, K, V, T_list)
    q = synth.normal_bf16((B, 16, 128), 122)
    idx, cnt = _select(np.random.default_rng(5), T_list, G, topk)
    cnt[3] = cnt[40] = 0
    good = _check_attention(sb, shape, layer, K, V, T_list, q, idx, cnt)
    bad, lens = idx.clone(), list(T_list)
    bad[7, 0, 0] = 64
    bad[8, 0, 0] = -2147483648
    bad[9, 0, 0] = 2147483647
    lens[20], lens[21] = 0, 4097
    out = torch.ones_like(good)
    sb.sparda_kv4_decode_attn(shape, layer, q.cuda(), bad, cnt, _i32(lens), B, out, sb.workspace(shape, B, sb.WS_KV4_ATTN))
    torch.cuda.synchronize()
    assert sb.sparda_device_error(clear=True) == sb.DEV_BAD_INDEX | sb.DEV_BAD_SEQ_LEN
    assert (out[20:22] == 0).all()
    same = [b for b in range(B) if b not in (7, 8, 9, 20, 21)]
    # the ranges per CTA moved with the lengths, and the order of the sums with them
    assert (out[same].float() - good[same].float()).abs().max() <= 2.0 ** -7 * good.float().abs().max()
    assert not torch.isnan(out).any()


def test_attention_many_blocks_nan_and_repeats(sb):
    T_list = [9000, 16000, 77, 16384, 333, 5000, 16384, 2]
    shape = sb.Shape(n_groups=2, heads_per_group=4, max_ctx=16384, max_batch=8)
    K, V = _kv(shape, 131)
    K[1, 1, 15990, 3] = float("nan")
    V[3, 0, 100, 64] = float("inf")
    layer = _filled(sb, shape, K, V, T_list)
    q = synth.normal_bf16((8, 8, 128), 132).cuda()
    ws = sb.workspace(shape, 8, sb.WS_KV4_ATTN)
    outs = []
    for _ in range(4):
        outs.append(torch.zeros((8, 8, 128), dtype=torch.bfloat16, device="cuda"))
        sb.sparda_kv4_decode_attn(shape, layer, q, None, None, _i32(T_list), 8, outs[-1], ws)
    torch.cuda.synchronize()
    assert sb.sparda_device_error(clear=True) == 0
    for o in outs[1:]:
        assert torch.equal(o.view(torch.int16), outs[0].view(torch.int16))
    nan = torch.isnan(outs[0])
    assert nan[1, 4:].all() and not nan[1, :4].any()
    assert nan[3, :4, 64:96].all() and not nan[3, :4, :64].any() and not nan[3, 4:].any()
    assert not nan[[0, 2, 4, 5, 6, 7]].any()


@pytest.mark.parametrize("fmt", ["kv4", "bf16"])
@pytest.mark.parametrize("B,topk", [(1, 62), (20, 30), (90, 14)])
def test_mass_of_repeated_blocks_is_reproducible(sb, fmt, B, topk):
    """Lists that name few blocks many times, over the CTAs of a cluster or of the planned form: the same
    bits in every call, and what the list's 64-bit reference adds up."""
    T, n = 1900, topk + 2
    shape = sb.Shape(n_groups=2, heads_per_group=16, max_ctx=1920, max_batch=B, topk=topk)
    K, V = _kv(shape, 81)
    T_list = [T] * B
    layer = _filled(sb, shape, K, V, T_list)
    if fmt == "bf16":
        layer = sb.LayerKV(K.cuda(), V.cuda(), torch.zeros_like(layer.ck))
    q = synth.normal_bf16((B, 32, 128), 82) * 2
    gen = torch.Generator().manual_seed(83)
    idx = torch.randint(0, 5, (B, 2, n), generator=gen, dtype=torch.int32) * 7
    cnt = torch.randint(1, n + 1, (B, 2), generator=gen, dtype=torch.int32)
    cnt[0] = n
    out = torch.empty((B, 32, 128), dtype=torch.bfloat16, device="cuda")
    kind, call = (sb.WS_KV4_ATTN_MASS, sb.sparda_kv4_decode_attn) if fmt == "kv4" else (
        sb.WS_ATTN_MASS, sb.sparda_sparse_decode_attn_mass)
    ws, seq, qd, di, dc = sb.workspace(shape, B, kind), _i32(T_list), q.cuda(), idx.cuda(), cnt.cuda()
    start = torch.rand((B, 2, 30), generator=gen).cuda()
    masses = []
    for _ in range(12):
        masses.append(start.clone())
        call(shape, layer, qd, di, dc, seq, B, out, ws, mass=masses[-1])
    torch.cuda.synchronize()
    assert sb.sparda_device_error(clear=True) == 0
    assert all(torch.equal(m, masses[0]) for m in masses[1:])
    k64 = R.grid_values(K, True) if fmt == "kv4" else to64(K)
    v64 = _v16(V) if fmt == "kv4" else to64(V)
    for b in (0, B - 1):
        for g in range(2):
            blocks = idx[b, g, :cnt[b, g]].tolist()
            _, _, w, tol = R.attention(to64(q)[b, 16 * g:16 * g + 16], k64[b, g], v64[b, g], blocks, T, W16)
            want = start[b, g].cpu().double().numpy()
            bound = 2.0 ** -22 * want
            for j, x in zip(blocks, w):
                want[j] += x
                bound[j] += tol * x + 2.0 ** -22 * want[j]
            assert (np.abs(masses[0][b, g].cpu().double().numpy() - want) <= bound).all()


def test_attention_joins_of_many_ctas(sb):
    """Groups that spread over more CTAs than join at once, beside short ones: exact, the same bits in every
    call, and every counter of the workspace left at zero."""
    T_list = [40000, 64, 1, 20000]
    shape = sb.Shape(n_groups=1, heads_per_group=7, max_ctx=40000, max_batch=4)
    K, V = _kv(shape, 95)
    layer = _filled(sb, shape, K, V, T_list)
    q = synth.normal_bf16((4, 7, 128), 96)
    _check_attention(sb, shape, layer, K, V, T_list, q, None, None, mass=True)
    ws = sb.workspace(shape, 4, sb.WS_KV4_ATTN)
    outs = []
    for _ in range(8):
        outs.append(torch.zeros((4, 7, 128), dtype=torch.bfloat16, device="cuda"))
        sb.sparda_kv4_decode_attn(shape, layer, q.cuda(), None, None, _i32(T_list), 4, outs[-1], ws)
    torch.cuda.synchronize()
    assert all(torch.equal(o, outs[0]) for o in outs[1:])
    assert (ws[:256 + 1280] == 0).all()              # the counters lie before the partial results
    assert sb.sparda_device_error(clear=True) == 0


@pytest.mark.parametrize("mass", [False, True])
@pytest.mark.parametrize("T_list,G,H,ctx,topk", [
    ([2200] * 70, 2, 16, 2240, 32),                # one CTA per group, whole blocks per warp
    ([1500, 90] * 40, 2, 5, 1536, 32),             # more groups than SMs, many blocks each: ranges over groups
    ([1400] * 100, 2, 8, 1408, 9),                 # more groups than SMs, few blocks each
    ([20000, 13000], 1, 16, 20032, 0),             # few groups, several warps per block
    ([20000, 13000], 1, 6, 20032, 0),
])
def test_attention_forms(sb, T_list, G, H, ctx, topk, mass):
    B = len(T_list)
    shape = sb.Shape(n_groups=G, heads_per_group=H, max_ctx=ctx, max_batch=B + 1, topk=max(1, topk))
    K, V = _kv(shape, 97)
    layer = _filled(sb, shape, K, V, T_list)
    q = synth.normal_bf16((B, G * H, 128), 98)
    idx = cnt = None
    if topk:
        idx, cnt = _select(np.random.default_rng(99), T_list, G, topk)
    _check_attention(sb, shape, layer, K, V, T_list, q, idx, cnt, mass=mass)


def test_attention_whole_groups_of_long_caches(sb):
    """More groups than the plan holds, in caches of more blocks than a cluster takes: whole groups per CTA."""
    B, ctx = 530, 1600
    shape = sb.Shape(n_groups=2, heads_per_group=9, max_ctx=ctx, max_batch=B)
    small = sb.Shape(n_groups=2, heads_per_group=9, max_ctx=ctx, max_batch=5)
    K, V = _kv(small, 101)
    T_list = [ctx if b % 97 == 0 else 1 + (37 * b) % 300 for b in range(B)]
    rep = [b % 5 for b in range(B)]
    layer = sb.LayerKV4.empty(shape)
    layer.kv.fill_(0xff)
    sb.sparda_kv4_quantize(shape, layer, K.cuda()[rep], V.cuda()[rep], _i32(T_list), B)
    q = synth.normal_bf16((B, 18, 128), 102)
    out = torch.empty((B, 18, 128), dtype=torch.bfloat16, device="cuda")
    mass = torch.zeros((B, 2, ctx // 64), device="cuda")
    ws = sb.workspace(shape, B, sb.WS_KV4_ATTN_MASS)
    sb.sparda_kv4_decode_attn(shape, layer, q.cuda(), None, None, _i32(T_list), B, out, ws, mass=mass)
    torch.cuda.synchronize()
    assert sb.sparda_device_error(clear=True) == 0
    k64, v64 = R.grid_values(K, True), _v16(V)
    for b in list(range(0, B, 23)) + [97, 194, B - 1]:
        for g in range(2):
            ref, tol, w, wtol = R.attention(to64(q)[b, 9 * g:9 * g + 9], k64[rep[b], g], v64[rep[b], g], None, T_list[b], W16)
            assert (np.abs(to64(out)[b, 9 * g:9 * g + 9] - ref) <= tol).all(), b
            got = mass[b, g].cpu().double().numpy()
            assert (np.abs(got[:len(w)] - w) <= wtol * w + 2.0 ** -22 * w).all() and (got[len(w):] == 0).all()
