"""The binding's own checks of the head norm and rotation's tensors, and the
library's refusals, which need no GPU: every one comes before a launch."""
import ctypes

import pytest
import torch

import tensor_transformer_layer_cube_gb300 as t

BF16 = torch.bfloat16
EINVAL, ESHAPE, EALIGN, EDTYPE, EUNSUP, EOVER = 1, 2, 3, 4, 7, 8


@pytest.fixture(scope="module", autouse=True)
def built():
    t.build()


def rope(d=64, r=64, dtype=BF16, **kw):
    kw = {"norm": True, "q_weight": torch.ones(d, dtype=dtype), "k_weight": torch.ones(d, dtype=dtype)} | kw
    turns = torch.zeros(max(r // 2, 1), dtype=torch.int64)
    x = t.rope(turns, dtype, d, r, **kw)
    x.keep = (turns, kw)
    return x


def rows(n=3, h=4, d=64, dtype=BF16):
    return torch.zeros(n, h, d, dtype=dtype)


POS = torch.zeros(8, dtype=torch.int32)


def test_descriptors():
    turns = torch.zeros(32, dtype=torch.int64)
    for bad in (dict(dtype=torch.float16), dict(turns=turns.int()), dict(turns=turns[:31]), dict(turns=None),
                dict(q_weight=torch.ones(64)), dict(k_weight=torch.ones(63, dtype=BF16)),
                dict(q_weight=torch.ones(128, dtype=BF16)[::2])):
        with pytest.raises(ValueError):
            t.rope(**(dict(turns=turns, dtype=BF16, head_dim=64, rotary_dim=64) | bad))


@pytest.mark.parametrize("bad", [dict(K=rows(2)), dict(Q_out=rows(3, 5)), dict(K_out=rows(d=128)),
                                 dict(Q=rows(dtype=torch.float32)), dict(K=rows(d=128)[..., ::2]),
                                 dict(positions=POS.long()), dict(positions=POS[:2]), dict(positions=POS[::2])])
def test_rows_and_positions(bad):
    a = dict(Q=rows(), K=rows(), positions=POS, Q_out=rows(), K_out=rows()) | bad
    with pytest.raises(ValueError):
        t.tp3d_qk_rope(None, rope(), **a, stream=0)


def test_rows_of_the_backward_and_the_store():
    r = rope()
    ok = dict(Q=rows(), K=rows(), positions=POS, dQ_out=rows(), dK_out=rows(), dQ=rows(), dK=rows(), dq_weight=None,
              dk_weight=None, workspace=None)
    for bad in (dict(dQ=rows(2)), dict(dK=rows(3, 2)), dict(Q=rows(3, 2)), dict(dq_weight=torch.ones(64)),
                dict(dk_weight=torch.ones(63, dtype=BF16))):
        with pytest.raises(ValueError):
            t.tp3d_qk_rope_bwd(None, r, **(ok | bad), stream=0)
    pool = torch.zeros(2, 16, 2, 64, dtype=BF16)
    cache = t.kv_cache(pool, torch.zeros_like(pool))
    ok = dict(Q=rows(), K=rows(3, 2), V=rows(3, 2), positions=POS, slots=torch.zeros(3, dtype=torch.int64), Q_out=rows())
    for bad in (dict(K=rows()), dict(V=rows(2, 2)), dict(slots=torch.zeros(3)), dict(slots=torch.zeros(2, dtype=torch.int64))):
        with pytest.raises(ValueError):
            t.tp3d_paged_rope_store(None, r, cache, **(ok | bad), stream=0)


class Fake:
    """A context's memory: what the host checks read of it is zero, and they refuse before anything else is used."""

    def __init__(self):
        self.mem = (ctypes.c_char * 4096)()
        self.at = ctypes.addressof(self.mem)


def buffer():
    x = torch.zeros((1 << 16) + 128, dtype=BF16)
    return x[-x.data_ptr() % 256 // 2:][:1 << 16]


def test_refusals_of_the_forward():
    fake, lib = Fake(), t.lib()
    buf = buffer()

    def call(r=None, n=3, h=4, kh=2, q=None, k=None, qo=None, ko=None, pos=POS.data_ptr(), ctx=fake.at, **kw):
        r = rope() if r is None else r
        for key, v in kw.items():
            setattr(r, key, v)
        base = buf.data_ptr()
        a = {"q": (base, 1024, 64), "k": (base + 16384, 1024, 64), "qo": (base + 32768, 1024, 64),
             "ko": (base + 65536, 1024, 64)}
        for key, v in (("q", q), ("k", k), ("qo", qo), ("ko", ko)):
            a[key] = v(*a[key]) if callable(v) else a[key]
        x = {key: [p, t.tp3d_row_strides(ts, hs)] for key, (p, ts, hs) in a.items()}
        return lib.tp3d_qk_rope(ctx, ctypes.byref(r), n, h, kh, *x["q"], *x["k"], pos, *x["qo"], *x["ko"], None)
    assert call(n=0) == 0
    assert call(ctx=None) == EINVAL and call(n=-1) == EINVAL and call(h=0) == EINVAL and call(kh=0) == EINVAL
    assert call(pos=None) == EINVAL and call(pos=POS.data_ptr() + 2) == EALIGN
    assert call(n=2 ** 31) == EUNSUP and call(h=65537) == EUNSUP
    for x in ("q", "k", "qo", "ko"):
        assert call(**{x: lambda p, a, b: (None, a, b)}) == EINVAL
        assert call(**{x: lambda p, a, b: (p, 0, b)}) == EINVAL and call(**{x: lambda p, a, b: (p, a, -64)}) == EINVAL
        assert call(**{x: lambda p, a, b: (p + 8, a, b)}) == EALIGN and call(**{x: lambda p, a, b: (p, a, 68)}) == EALIGN
        assert call(**{x: lambda p, a, b: (p, 1 << 39, b)}) == EUNSUP
    assert call(dtype=2) == EDTYPE and call(head_dim=0) == EINVAL and call(rotary_dim=-16) == EINVAL
    assert call(head_dim=60, rotary_dim=0) == EUNSUP and call(head_dim=264) == EUNSUP and call(rotary_dim=24) == EUNSUP
    assert call(rotary_dim=80) == ESHAPE and call(norm=2) == EINVAL and call(interleaved=2) == EINVAL
    assert call(magnitude=float("nan")) == EINVAL and call(eps=-1.0) == EINVAL and call(eps=float("inf")) == EINVAL
    assert call(turns=None) == EINVAL and call(turns=buf.data_ptr() + 4) == EALIGN
    assert call(q_weight=buf.data_ptr() + 8) == EALIGN
    base = buf.data_ptr()
    assert call(qo=lambda p, a, b: (base, a, 128)) == EOVER  # the input's rows with other strides
    assert call(qo=lambda p, a, b: (base + 16, a, b)) == EOVER and call(ko=lambda p, a, b: (base, a, b)) == EOVER
    assert call(qo=lambda p, a, b: (base + 16384, a, b)) == EOVER  # query rows over the keys
    assert call(qo=lambda p, a, b: (base + 65536, a, b)) == EOVER  # two outputs
    assert call(pos=base + 32768) == EOVER and call(turns=base + 32768) == EOVER and call(k_weight=base + 65536) == EOVER
    # parts of the same rows that touch: 4 heads of 64 columns in rows of 320
    assert call(q=lambda p, a, b: (base, 320, 64), qo=lambda p, a, b: (base, 320, 64),
                k=lambda p, a, b: (base + 480, 320, 64)) == EOVER
    # a rotation without columns or a norm without weights refuses nothing by itself
    assert call(n=0, rotary_dim=0, turns=None, q_weight=None, k_weight=None) == 0


def test_refusals_of_the_backward():
    fake, lib = Fake(), t.lib()
    buf = buffer()
    base = buf.data_ptr()

    def call(n=3, r=None, ctx=fake.at, w=(base + 98304, base + 98560), ws=base + 100352, pos=POS.data_ptr(), **kw):
        r = rope() if r is None else r
        at = {"q": base, "k": base + 8192, "gq": base + 16384, "gk": base + 32768, "dq": base + 49152, "dk": base + 65536}
        at |= kw
        s = t.tp3d_row_strides(256, 64)
        x = {k: [p, s] for k, p in at.items()}
        return lib.tp3d_qk_rope_bwd(ctx, ctypes.byref(r), n, 4, 2, *x["q"], *x["k"], pos, *x["gq"], *x["gk"], *x["dq"],
                                    *x["dk"], *w, ws, None)
    assert call(ctx=None) == EINVAL and call(n=-1) == EINVAL and call(pos=None) == EINVAL
    for x in ("q", "k", "gq", "gk", "dq", "dk"):
        assert call(**{x: None}) == EINVAL and call(**{x: base + 8}) == EALIGN
    assert call(r=rope(norm=False)) == EINVAL  # weights' gradients without a norm
    assert call(ws=None) == EINVAL and call(ws=base + 100352 + 16) == EALIGN and call(w=(base + 98312, None)) == EALIGN
    assert call(dq=base) == EOVER and call(dk=base + 16384) == EOVER and call(dk=base + 49152) == EOVER
    assert call(w=(base + 98304, base + 98304)) == EOVER and call(w=(base + 49152, None)) == EOVER
    assert call(pos=base + 49152) == EOVER and call(pos=base + 98304) == EOVER
    assert call(n=0, w=(None, None), ws=None) == 0


def test_refusals_of_the_store():
    fake, lib = Fake(), t.lib()
    buf = buffer()
    base = buf.data_ptr()
    kp, vp = torch.zeros(2, 16, 2, 64, dtype=BF16), torch.zeros(2, 16, 2, 64, dtype=BF16)
    slots = torch.zeros(8, dtype=torch.int64)

    def call(n=3, h=4, r=None, ctx=fake.at, pos=POS.data_ptr(), sl=slots.data_ptr(), cache=None, **kw):
        r = rope() if r is None else r
        c = t.kv_cache(kp, vp) if cache is None else cache
        at = {"q": base, "k": base + 8192, "v": base + 16384, "qo": base + 32768} | kw
        s = t.tp3d_row_strides(256, 64)
        x = {k: [p, s] for k, p in at.items()}
        return lib.tp3d_paged_rope_store(ctx, ctypes.byref(r), ctypes.byref(c), n, h, *x["q"], *x["k"], *x["v"], pos, sl,
                                         *x["qo"], None)
    assert call(n=0) == 0
    assert call(ctx=None) == EINVAL and call(n=-1) == EINVAL and call(h=0) == EINVAL
    assert call(pos=None) == EINVAL and call(sl=None) == EINVAL and call(sl=slots.data_ptr() + 4) == EALIGN
    for x in ("q", "k", "v", "qo"):
        assert call(**{x: None}) == EINVAL and call(**{x: base + 8}) == EALIGN
        assert call(**{x: vp.data_ptr()}) == EOVER
    assert call(qo=base + 8192) == EOVER and call(qo=base + 16384) == EOVER and call(qo=base + 16) == EOVER
    assert call(pos=kp.data_ptr()) == EOVER and call(sl=kp.data_ptr()) == EOVER and call(sl=base + 32768) == EOVER
    assert call(r=rope(d=128, r=64)) == ESHAPE
    r = rope(dtype=torch.float32)
    assert call(r=r) == EDTYPE
    c = t.kv_cache(kp, vp)
    c.dtype = t.TP3D_F32
    assert call(r=r, cache=c) == EDTYPE
