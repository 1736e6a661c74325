"""Host-side checks of the 4-bit cache, block-mass and eviction entry points: workspace sizes and
every refusal, all before any launch (no GPU needed)."""
import ctypes

import pytest
import torch

from block_sparse_attention_forecast_gb300 import build as _build

_build.build()

import block_sparse_attention_forecast_gb300.binding as sb  # noqa: E402

P = ctypes.c_void_p
FAKE, FAKE2, ODD = P(1 << 20), P(1 << 24), P((1 << 20) + 8)
BIG = 1 << 40


def _shape(**kw):
    return sb.Shape(**{**dict(max_batch=2, max_ctx=4096, topk=8), **kw})


def _ref(s):
    return ctypes.byref(s.c())


def _l4(kv=1 << 20, ck=1 << 20):
    return ctypes.byref(sb.c_layer_kv4(kv, ck))


def _lk(k=1 << 20, v=1 << 20, ck=1 << 20, on_host=0):
    return ctypes.byref(sb.c_layer_kv(k, v, ck, None, None, on_host, 0))


def test_workspace_sizes():
    for H in (1, 5, 16):
        s = _shape(heads_per_group=H)
        plain = sb.sparda_workspace_bytes(s, 2, sb.WS_KV4_ATTN)
        mass = sb.sparda_workspace_bytes(s, 2, sb.WS_KV4_ATTN_MASS)
        # counters, then two partial results for each of at least 152 CTAs
        assert plain >= 2 * 2 * 4 + 152 * 2 * (16 * 128 + 32) * 4
        # statistics of every block (64 of them here, more than the 10 selectable ones)
        assert mass >= plain + 2 * 2 * 64 * 4 * 16 * 8 + 2 * 2 * 2 * 16 * 4
    assert sb.sparda_workspace_bytes(_shape(heads_per_group=17), 2, sb.WS_KV4_ATTN) == 0
    assert sb.sparda_workspace_bytes(_shape(heads_per_group=0), 2, sb.WS_KV4_ATTN) == 0
    assert sb.sparda_workspace_bytes(_shape(), 3, sb.WS_KV4_ATTN) == 0
    attn = sb.sparda_workspace_bytes(_shape(), 2, sb.WS_ATTN)
    assert sb.sparda_workspace_bytes(_shape(), 2, sb.WS_ATTN_MASS) >= attn + 2 * 2 * 10 * 4 * 16 * 8
    assert sb.sparda_workspace_bytes(_shape(heads_per_group=8), 2, sb.WS_ATTN_MASS) == 0


def test_cache_calls_reject_bad_arguments():
    s = _ref(_shape())
    for fn in (sb.lib.sparda_kv4_quantize, sb.lib.sparda_kv4_append):
        assert fn(None, _l4(), FAKE, FAKE, FAKE, 1, None) == sb.ERR_INVALID_ARG
        assert fn(_ref(_shape(heads_per_group=17)), _l4(), FAKE, FAKE, FAKE, 1, None) == sb.ERR_UNSUPPORTED_SHAPE
        assert fn(_ref(_shape(head_dim=64)), _l4(), FAKE, FAKE, FAKE, 1, None) == sb.ERR_UNSUPPORTED_SHAPE
        assert fn(s, None, FAKE, FAKE, FAKE, 1, None) == sb.ERR_INVALID_ARG
        assert fn(s, _l4(kv=None), FAKE, FAKE, FAKE, 1, None) == sb.ERR_INVALID_ARG
        assert fn(s, _l4(kv=(1 << 20) + 8), FAKE, FAKE, FAKE, 1, None) == sb.ERR_MISALIGNED
        assert fn(s, _l4(), None, FAKE, FAKE, 1, None) == sb.ERR_INVALID_ARG
        assert fn(s, _l4(), FAKE, None, FAKE, 1, None) == sb.ERR_INVALID_ARG
        assert fn(s, _l4(), FAKE, FAKE, None, 1, None) == sb.ERR_INVALID_ARG
        assert fn(s, _l4(), ODD, FAKE, FAKE, 1, None) == sb.ERR_MISALIGNED
        assert fn(s, _l4(), FAKE, ODD, FAKE, 1, None) == sb.ERR_MISALIGNED
        assert fn(s, _l4(), FAKE, FAKE, FAKE, 0, None) == sb.ERR_INVALID_ARG
        assert fn(s, _l4(), FAKE, FAKE, FAKE, 3, None) == sb.ERR_INVALID_ARG
    # only the append needs the compressed keys
    assert sb.lib.sparda_kv4_append(s, _l4(ck=None), FAKE, FAKE, FAKE, 1, None) == sb.ERR_INVALID_ARG
    deq = sb.lib.sparda_kv4_dequantize
    assert deq(s, _l4(), FAKE, None, FAKE, 1, FAKE, FAKE, None) == sb.ERR_INVALID_ARG       # idx without cnt
    assert deq(s, _l4(), None, FAKE, FAKE, 1, FAKE, FAKE, None) == sb.ERR_INVALID_ARG
    assert deq(s, _l4(), P(2), FAKE, FAKE, 1, FAKE, FAKE, None) == sb.ERR_MISALIGNED
    assert deq(s, _l4(), None, None, FAKE, 1, None, FAKE, None) == sb.ERR_INVALID_ARG


def test_attention_rejects_bad_arguments():
    s = _shape()
    need, need_mass = (sb.sparda_workspace_bytes(s, 2, k) for k in (sb.WS_KV4_ATTN, sb.WS_KV4_ATTN_MASS))

    def call(shape=s, layer=None, q=FAKE, idx=FAKE, cnt=FAKE, seq=FAKE, batch=1, out=FAKE, mass=None, ws=FAKE, n=BIG):
        return sb.lib.sparda_kv4_decode_attn(_ref(shape), layer or _l4(ck=None), q, idx, cnt, seq, batch, out, mass, ws,
                                             n, None)
    assert call(shape=_shape(heads_per_group=17)) == sb.ERR_UNSUPPORTED_SHAPE
    assert call(shape=_shape(topk=63)) == sb.ERR_UNSUPPORTED_SHAPE
    assert call(layer=_l4(kv=None)) == sb.ERR_INVALID_ARG
    for name in ("q", "seq", "out", "ws"):
        assert call(**{name: None}) == sb.ERR_INVALID_ARG, name
    assert call(idx=None) == sb.ERR_INVALID_ARG and call(cnt=None) == sb.ERR_INVALID_ARG
    for name in ("q", "out", "ws"):
        assert call(**{name: ODD}) == sb.ERR_MISALIGNED, name
    assert call(mass=P(2)) == sb.ERR_MISALIGNED
    assert call(batch=3) == sb.ERR_INVALID_ARG
    assert call(n=need - 1) == sb.ERR_WORKSPACE_TOO_SMALL
    assert call(mass=FAKE, n=need_mass - 1) == sb.ERR_WORKSPACE_TOO_SMALL
    m = sb.lib.sparda_sparse_decode_attn_mass
    assert m(_ref(s), _lk(), FAKE, FAKE, FAKE, FAKE, 1, FAKE, None, FAKE, BIG, None) == sb.ERR_INVALID_ARG
    assert m(_ref(s), _lk(on_host=1), FAKE, FAKE, FAKE, FAKE, 1, FAKE, FAKE, FAKE, BIG, None) == sb.ERR_INVALID_ARG
    assert m(_ref(s), _lk(), FAKE, FAKE, FAKE, FAKE, 1, FAKE, P(2), FAKE, BIG, None) == sb.ERR_MISALIGNED
    assert m(_ref(_shape(heads_per_group=8)), _lk(), FAKE, FAKE, FAKE, FAKE, 1, FAKE, FAKE, FAKE, BIG,
             None) == sb.ERR_UNSUPPORTED_SHAPE


@pytest.mark.parametrize("kv4", [False, True])
def test_eviction_rejects_bad_arguments(kv4):
    s = _shape()
    fn = sb.lib.sparda_kv4_evict_blocks if kv4 else sb.lib.sparda_evict_blocks
    layer = _l4 if kv4 else _lk
    other = (lambda **k: _l4(**{**dict(kv=1 << 24, ck=1 << 24), **k})) if kv4 else \
            (lambda **k: _lk(**{**dict(k=1 << 24, v=1 << 24, ck=1 << 24), **k}))

    def call(shape=s, L=None, mass=FAKE, seq=FAKE, ds=None, dl=None, dm=None, dq=None, batch=1, keep=8, recent=2, kept=FAKE):
        return fn(_ref(shape), L or layer(), mass, seq, None if ds is None else _ref(ds), dl, dm, dq, batch, keep, recent,
                  kept, None)
    assert call(mass=None) == sb.ERR_INVALID_ARG and call(seq=None) == sb.ERR_INVALID_ARG
    assert call(kept=None) == sb.ERR_INVALID_ARG and call(batch=3) == sb.ERR_INVALID_ARG
    assert call(recent=0) == sb.ERR_INVALID_ARG and call(keep=2, recent=2) == sb.ERR_INVALID_ARG
    assert call(keep=4097) == sb.ERR_UNSUPPORTED_SHAPE
    assert call(L=layer(ck=None)) == sb.ERR_INVALID_ARG
    assert call(mass=P(2)) == sb.ERR_MISALIGNED and call(kept=P(2)) == sb.ERR_MISALIGNED
    full = dict(ds=s, dl=other(), dm=FAKE2, dq=FAKE2)
    for name in full:
        assert call(**{**full, name: None}) == sb.ERR_INVALID_ARG, name
    assert call(**{**full, "dl": layer()}) == sb.ERR_INVALID_ARG                    # the source itself
    assert call(**{**full, "dm": FAKE}) == sb.ERR_INVALID_ARG
    assert call(**{**full, "dq": FAKE}) == sb.ERR_INVALID_ARG
    assert call(**{**full, "dl": other(ck=1 << 20)}) == sb.ERR_INVALID_ARG
    assert call(**{**full, "ds": _shape(max_ctx=256)}) == sb.ERR_UNSUPPORTED_SHAPE  # 4 blocks for 8
    assert call(**{**full, "ds": _shape(n_groups=1)}) == sb.ERR_UNSUPPORTED_SHAPE
    assert call(**{**full, "ds": _shape(max_batch=1)}, batch=2) == sb.ERR_UNSUPPORTED_SHAPE
    assert call(**{**full, "dl": other(ck=(1 << 24) + 8)}) == sb.ERR_MISALIGNED
    if not kv4:
        assert call(L=_lk(on_host=1)) in (sb.ERR_INVALID_ARG, sb.ERR_NOT_MAPPED_HOST)
        assert call(shape=_shape(heads_per_group=8)) == sb.ERR_UNSUPPORTED_SHAPE


def test_binding_refuses_tensors_on_another_device():
    s = _shape()
    cpu = sb.LayerKV4.empty(s, device="cpu")
    assert cpu.kv.shape == (2, 2, 64, sb.KV4_BLOCK_BYTES) and cpu.ck.shape == (2, 2, 255, 128)
    seq = torch.ones(2, dtype=torch.int32)
    x = torch.zeros((2, 2, 128), dtype=torch.bfloat16)
    with pytest.raises((ValueError, RuntimeError)):
        sb.sparda_kv4_append(s, cpu, x, x, seq, 2)


def test_binding_checks_types_sizes_and_strides():
    dev = -1
    ok = torch.zeros((4, 8), dtype=torch.bfloat16)
    assert sb._checked("x", ok, torch.bfloat16, 32, dev) == ok.data_ptr()
    for bad in (ok.float(), ok[:3], ok.t()):
        with pytest.raises(ValueError):
            sb._checked("x", bad, torch.bfloat16, 32, dev)


@pytest.mark.parametrize("kv4", [False, True])
def test_eviction_refuses_a_destination_inside_the_source(kv4):
    """A destination that shares any memory with the source, not its first byte only."""
    s, base = _shape(max_batch=2, n_groups=2, max_ctx=1024), 1 << 30
    fn = sb.lib.sparda_kv4_evict_blocks if kv4 else sb.lib.sparda_evict_blocks
    plane = 4 * (16 * 10240 if kv4 else 1024 * 256)
    ck = 4 * sb.num_windows(1024) * 256
    if kv4:
        make = lambda k, v, c: _l4(kv=k, ck=c)
    else:
        make = lambda k, v, c: _lk(k=k, v=v, ck=c)
    far = base << 4
    src = make(base, base + plane, base + 2 * plane)

    def call(k=far, v=far + plane, c=far + 2 * plane, mass=1 << 20, dm=1 << 21, seq=1 << 22, dq=1 << 23, batch=2, keep=8):
        return fn(_ref(s), src, P(mass), P(seq), _ref(s), make(k, v, c), P(dm), P(dq), batch, keep, 2, P(1 << 25), None)
    bad = sb.ERR_INVALID_ARG
    assert call(k=base + 16) == bad and call(k=base + plane - 16) == bad and call(k=base - plane + 16) == bad
    assert call(c=base + 2 * plane + ck - 16) == bad                       # compressed keys
    assert call(c=base + 16) == bad and call(k=base + 2 * plane + 16) == bad      # of different kinds
    assert call(dm=(1 << 20) + 4) == bad and call(dq=(1 << 22) + 4) == bad
    if not kv4:
        assert call(v=base + 32) == bad and call(k=base + plane + 64) == bad
    # side by side is apart: no refusal of the arguments
    for ok in (dict(), dict(c=base + 2 * plane + ck), dict(dq=(1 << 22) + 8), dict(dm=(1 << 20) + 4 * 64)):
        assert call(**ok, keep=4097) == sb.ERR_UNSUPPORTED_SHAPE
        if not torch.cuda.is_available():
            assert call(**ok) != bad


def test_layers_are_checked_again_when_a_field_changes():
    """The C struct kept with a layer goes when a field is set, and with a pickle or a copy."""
    import copy
    import pickle
    shape = sb.Shape(max_batch=1, n_groups=1, max_ctx=64)
    for layer, field in ((sb.LayerKV(torch.zeros(1, 1, 64, 128), torch.zeros(1, 1, 64, 128), torch.zeros(1, 1, 3, 128)), "k"),
                         (sb.LayerKV4.empty(shape, device="cpu"), "kv")):
        layer.__dict__["_args"] = (1, 2, ctypes.byref(ctypes.c_int(0)))
        assert "_args" not in pickle.loads(pickle.dumps(layer)).__dict__
        assert "_args" not in copy.copy(layer).__dict__ and "_args" not in copy.deepcopy(layer).__dict__
        assert "_args" in layer.__dict__
        setattr(layer, field, getattr(layer, field).clone())
        assert "_args" not in layer.__dict__
    n = shape.sizes()
    shape.max_batch = 3
    assert shape.sizes() == tuple(3 * x for x in n) and pickle.loads(pickle.dumps(shape)) == shape


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("batch", [1, 3])
def test_eviction_takes_weights_of_the_batch_alone(kv4, batch):
    """Weight arrays of `batch` sequences, fewer than max_batch, directly side by side: they are apart, on
    either side, and one float nearer they are not."""
    s, d = _shape(max_batch=8, n_groups=2, max_ctx=1024), _shape(max_batch=4, n_groups=2, max_ctx=512)
    fn = sb.lib.sparda_kv4_evict_blocks if kv4 else sb.lib.sparda_evict_blocks
    src, dst = (_l4(kv=1 << 34, ck=1 << 33), _l4(kv=1 << 36, ck=1 << 35)) if kv4 else \
        (_lk(k=1 << 34, v=1 << 37, ck=1 << 33), _lk(k=1 << 36, v=1 << 38, ck=1 << 35))
    m = 1 << 20
    n_src, n_dst = batch * 2 * 16 * 4, batch * 2 * 8 * 4           # bytes of the two arrays

    def call(mass, dm):
        return fn(_ref(s), src, P(mass), P(1 << 22), _ref(d), dst, P(dm), P(1 << 23), batch, 8, 2, P(1 << 25), None)
    assert call(m, m + n_src - 4) == sb.ERR_INVALID_ARG and call(m, m - n_dst + 4) == sb.ERR_INVALID_ARG
    if not torch.cuda.is_available():              # (made-up addresses: not where the call could launch)
        for dm in (m + n_src, m - n_dst):
            assert call(m, dm) == sb.ERR_CUDA


def test_what_a_shape_keeps_is_no_field():
    """A shape that calls have used is copied, spread and compared as one that they have not."""
    import copy
    import dataclasses
    import pickle
    used, fresh = _shape(), _shape()
    used.ref(), used.sizes()
    assert vars(used) == vars(fresh) == dataclasses.asdict(fresh) and used == fresh and repr(used) == repr(fresh)
    for other in (sb.Shape(**vars(used)), sb.Shape(**{**vars(used), "max_batch": 3}), copy.copy(used), copy.deepcopy(used),
                  pickle.loads(pickle.dumps(used)), dataclasses.replace(used, topk=4)):
        assert other.sizes()[0] == other.max_batch * 2 * 4096 * 128
        got = other.ref()._obj
        assert (got.max_batch, got.topk) == (other.max_batch, other.topk)
        other.max_batch += 1                       # what it keeps is its own
        assert other.ref()._obj.max_batch == other.max_batch and other.sizes()[0] == other.max_batch * 2 * 4096 * 128
    assert used.ref()._obj.max_batch == 2
    with pytest.raises(AttributeError):
        used.w_cap = 5                             # follows from the fields


@pytest.mark.parametrize("kv4", [False, True])
def test_eviction_refuses_lists_past_32_bits(kv4):
    """keep may exceed a cache's blocks, so kept can be larger than any cache: entries are counted in 32 bits."""
    fn = sb.lib.sparda_kv4_evict_blocks if kv4 else sb.lib.sparda_evict_blocks
    layer = _l4(kv=1 << 34, ck=1 << 33) if kv4 else _lk(k=1 << 34, v=1 << 37, ck=1 << 33)

    def call(max_batch, G, keep):
        s = _shape(max_batch=max_batch, n_groups=G, max_ctx=64)
        return fn(_ref(s), layer, P(1 << 20), P(1 << 22), None, None, None, None, max_batch, keep, 2, P(1 << 25), None)
    for big in ((1 << 18, 2, 4096), (1 << 17, 1, 4096), ((1 << 18) + 1, 8, 256)):
        assert call(*big) == sb.ERR_UNSUPPORTED_SHAPE, big
    if not torch.cuda.is_available():
        assert call((1 << 17) - 1, 1, 4096) == sb.ERR_CUDA
