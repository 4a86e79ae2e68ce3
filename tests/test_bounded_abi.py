"""Host validation of the bounded cache's calls (CPU: every case is rejected before any CUDA call) and the
binding's own checks."""
import ctypes

import pytest

import dsa_sparse_mla_paged_gb300 as dsa

FAKE = 0x10000  # never dereferenced: validation fails before any CUDA call
INVALID, UNSUPPORTED, WORKSPACE = dsa.DSA_ERR_INVALID, dsa.DSA_ERR_UNSUPPORTED, dsa.DSA_ERR_WORKSPACE


def _params(**kw):
    base = dict(batch=2, n_q=2, max_pages_per_req=10, num_pages=20, key_page_stride=8448, lat_page_stride=36864)
    base.update(kw)
    return dsa.make_params(**base)


def _call(fn, p, args, /, **change):
    args = {**args, "ws": FAKE, "bytes": dsa.workspace_size(p), **change}
    return getattr(dsa.load(), fn)(ctypes.byref(p), *args.values(), None)


def _dims(**kw):
    base = dict(q_nope_row=49152, q_nope_head=512, q_rope_row=6144, q_rope_head=64, c_kv_row=576, k_rope_row=576, eps=1e-6,
                interleaved=1)
    return dsa.LatentDims(**{**base, **kw})


def _front(p=None, dims=None, **change):
    args = dict(qn=FAKE, qr=FAKE, gq=FAKE, c=FAKE, kr=FAKE, gk=FAKE, freq=FAKE, pos=FAKE, lat=FAKE, table=FAKE, ctx=FAKE, out=FAKE)
    args = {**args, "ws": FAKE, "bytes": 256, **change}
    d = _dims() if dims is None else dims
    return dsa.load().dsa_latent_frontend(ctypes.byref(p or _params()), ctypes.byref(d), *args.values(), None)


@pytest.mark.parametrize("change", [
    dict(qn=None), dict(qn=FAKE + 8), dict(qr=None), dict(qr=FAKE + 2), dict(gq=FAKE + 8), dict(c=FAKE + 2), dict(kr=None),
    dict(kr=FAKE + 8), dict(gk=None), dict(gk=FAKE + 2), dict(freq=None), dict(freq=FAKE + 4), dict(pos=FAKE + 2), dict(lat=None),
    dict(lat=FAKE + 8), dict(table=None), dict(ctx=None), dict(out=FAKE + 8), dict(out=None, c=None), dict(ws=None),
    dict(ws=FAKE + 4)])
def test_latent_frontend_rejects(lib, change):
    assert _front(**change) == INVALID


@pytest.mark.parametrize("dims", [
    dict(q_nope_row=0), dict(q_nope_head=504), dict(q_nope_head=516), dict(q_rope_row=60), dict(q_rope_head=-64), dict(c_kv_row=0),
    dict(c_kv_row=577), dict(k_rope_row=56), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(interleaved=2), dict(q_nope_row=1 << 41)])
def test_latent_frontend_rejects_strides(lib, dims):
    assert _front(dims=_dims(**dims)) == INVALID


def test_latent_frontend_parts(lib):
    assert _front(bytes=255) == WORKSPACE
    # what a part does not use may be missing, or anything
    assert _front(qn=None, qr=None, gq=None, out=None, bytes=0, dims=_dims(q_nope_row=0, q_rope_head=1)) == WORKSPACE
    assert _front(c=None, kr=None, gk=None, lat=None, table=None, bytes=0, dims=_dims(c_kv_row=0, k_rope_row=0)) == WORKSPACE
    assert _front(gq=None, pos=None, bytes=0) == WORKSPACE
    assert dsa.load().dsa_latent_frontend(ctypes.byref(_params()), None, *[FAKE] * 12, FAKE, 256, None) == INVALID


WINDOW = dict(q=FAKE, lat=FAKE, sinks=4, window=100, table=FAKE, ctx=FAKE, out=FAKE, lse=None)
MASS = dict(q=FAKE, lat=FAKE, sinks=4, window=100, table=FAKE, ctx=FAKE, lse=FAKE, fresh=2, mass=FAKE, stride=640)


@pytest.mark.parametrize("fn,args", [("dsa_window_mla_decode", WINDOW), ("dsa_attention_mass", MASS)])
@pytest.mark.parametrize("change", [
    dict(q=None), dict(q=FAKE + 2), dict(lat=FAKE + 8), dict(lat=None), dict(sinks=-1), dict(window=0), dict(window=-5),
    dict(table=None), dict(ctx=None), dict(lse=FAKE + 2), dict(ws=None), dict(ws=FAKE + 4)])
def test_window_calls_reject(lib, fn, args, change):
    assert _call(fn, _params(), args, **change) == INVALID


def test_window_calls_limits(lib):
    p, top = _params(), (1 << 31) - 1
    assert _call("dsa_window_mla_decode", p, WINDOW, out=None) == INVALID
    assert _call("dsa_window_mla_decode", p, WINDOW, out=FAKE + 8) == INVALID
    assert _call("dsa_window_mla_decode", p, WINDOW, sinks=top, window=top, bytes=0) == WORKSPACE
    for change in (dict(lse=None), dict(fresh=-1), dict(mass=None), dict(mass=FAKE + 2), dict(stride=639)):
        assert _call("dsa_attention_mass", p, MASS, **change) == INVALID, change
    assert _call("dsa_attention_mass", p, MASS, fresh=top, bytes=dsa.workspace_size(p) - 1) == WORKSPACE
    big = _params(batch=1, n_q=65535, max_pages_per_req=1 << 22, topk=1)
    assert _call("dsa_window_mla_decode", big, WINDOW) == UNSUPPORTED
    assert _call("dsa_attention_mass", big, MASS, stride=1 << 28) == UNSUPPORTED


EVICT = dict(budgets=FAKE, sinks=4, recent=8, mass=FAKE, stride=640, pools=None, n=0, table=FAKE, ctx=FAKE, refs=FAKE, kept=None)


@pytest.mark.parametrize("change", [
    dict(budgets=None), dict(sinks=-1), dict(recent=-1), dict(mass=None), dict(mass=FAKE + 2), dict(stride=639), dict(table=None),
    dict(ctx=None), dict(refs=None), dict(kept=FAKE + 2), dict(n=-1), dict(n=1), dict(ws=None), dict(ws=FAKE + 8)])
def test_evict_rejects(lib, change):
    assert _call("dsa_tokens_evict", _params(), EVICT, **change) == INVALID


def test_evict_pools(lib):
    p, K, V = _params(), dsa.DSA_TOKEN_KEY_FP8, dsa.DSA_TOKEN_LAT_FP8

    def status(*pools, **kw):
        q, n = dsa.make_token_pools(pools)
        return _call("dsa_tokens_evict", p, EVICT, pools=q, n=n, **kw)

    good = (FAKE, V, 1, 0, 36864)
    assert status(good, bytes=0) == WORKSPACE
    assert status((FAKE, V, 3, 36864, 3 * 36864), (2 * FAKE, K, 2, 20 * 8448, 8448), bytes=0) == WORKSPACE
    assert status(good, (2 * FAKE, V, 1, 0, 36864), good) == INVALID  # its tokens would move twice
    for bad in ((None, V, 1, 0, 36864), (FAKE + 8, V, 1, 0, 36864), (FAKE, 4, 1, 0, 36864), (FAKE, -1, 1, 0, 36864),
                (FAKE, V, 0, 0, 36864), (FAKE, V, 1, 0, 36848), (FAKE, V, 1, 0, 36872), (FAKE, K, 1, 0, 8432),
                (FAKE, V, 2, 36864, 36864), (FAKE, V, 2, 36848, 1 << 20), (FAKE, V, 2, 36872, 1 << 20),
                (FAKE, V, 3, 36864, 3 * 36864 - 16), (FAKE, K, 2, 20 * 8448 - 16, 8448)):
        assert status((4 * FAKE, V, 1, 0, 36864), bad) == INVALID, bad
    assert status((FAKE, V, 4097, 36864, 1 << 30)) == UNSUPPORTED
    assert status((FAKE, V, 1, 0, 1 << 41)) == UNSUPPORTED
    far = _params(num_pages=1 << 30)  # pages at products past 63 bits
    q, n = dsa.make_token_pools([(FAKE, V, 2, 36864, 1 << 34)])
    assert _call("dsa_tokens_evict", far, EVICT, pools=q, n=n, bytes=0) == UNSUPPORTED
    many = [(FAKE * (i + 1), V, 1, 0, 36864) for i in range(65)]
    assert status(*many) == UNSUPPORTED
    assert status(*many[:64], bytes=0) == WORKSPACE
    p = _params(num_pages=(1 << 30) + 1)
    assert status(good) == UNSUPPORTED


def test_null_and_bad_params(lib):
    for fn, args in (("dsa_window_mla_decode", WINDOW), ("dsa_attention_mass", MASS), ("dsa_tokens_evict", EVICT)):
        f = getattr(lib, fn)
        assert f(None, *args.values(), FAKE, 0, None) == INVALID, fn
        p = _params()
        p.batch = 0
        assert f(ctypes.byref(p), *args.values(), FAKE, 0, None) == INVALID, fn
        p = _params()
        p.heads = 64
        assert f(ctypes.byref(p), *args.values(), FAKE, 0, None) == UNSUPPORTED, fn
    p = _params()
    p.n_q = 0
    assert _front(p) == INVALID


def test_binding_checks():
    import torch

    bf, p = torch.bfloat16, _params()
    z = lambda *s, dtype=bf: torch.zeros(s, dtype=dtype)
    ok = dict(q_nope=z(4, 96, 512), q_rope=z(4, 96, 192)[:, :, 128:], gamma_q=None, c_kv=z(4, 576)[:, :512], k_rope=z(4, 576)[:, 512:],
              gamma_kv=z(512), inv_freq=z(32, dtype=torch.float32), positions=None, lat_pool=FAKE, block_table=FAKE, ctx_lens=FAKE,
              q_out=z(4, 96, 576), ws=z(128, dtype=torch.uint8), stream=0)
    with pytest.raises(dsa.DSAError) as e:  # every tensor passes: the workspace is too small (or not aligned)
        dsa.latent_frontend(p, **ok)
    assert e.value.status in (WORKSPACE, INVALID)
    for name, bad in (("q_nope", z(4, 96, 512, dtype=torch.float16)), ("q_nope", z(3, 96, 512)), ("q_nope", z(4, 512, 96).transpose(1, 2)),
                      ("q_nope", z(4, 95, 512)), ("q_nope", z(2, 3, 96, 512)[:, :2]), ("q_rope", z(4, 96, 32)), ("c_kv", z(4, 512, dtype=torch.float32)),
                      ("c_kv", z(5, 512)), ("k_rope", z(4, 128)[:, ::2]), ("gamma_kv", z(511)), ("gamma_q", z(1024)[::2]),
                      ("inv_freq", z(32)), ("positions", z(4, dtype=torch.int64)), ("positions", z(3, dtype=torch.int32)),
                      ("q_out", z(3, 96, 576)), ("q_out", z(4, 96, 640)[:, :, :576])):
        with pytest.raises(ValueError, match=name):
            dsa.latent_frontend(p, **{**ok, name: bad})
    f32, i32 = torch.float32, torch.int32
    lse, mass = z(4, 96, dtype=f32), z(2, 640, dtype=f32)
    for name, bad in (("mass", z(2, 640)), ("mass", z(1, 640, dtype=f32)), ("mass", z(2, 639, dtype=f32)), ("mass", z(640, 2, dtype=f32).T),
                      ("mass", z(1, 640, dtype=f32).expand(2, 640)), ("lse", z(3, 96, dtype=f32)), ("lse", z(4, 96, dtype=torch.float64))):
        a = {"lse": lse, "mass": mass, name: bad}
        with pytest.raises(ValueError, match=name):
            dsa.attention_mass(p, FAKE, FAKE, 0, 640, FAKE, FAKE, a["lse"], 0, a["mass"], z(256, dtype=torch.uint8), 0)
    pools, budgets, ws = dsa.make_token_pools([]), z(2, dtype=i32), z(256, dtype=torch.uint8)
    for v in (1 << 31, (1 << 32) + 5, 1 << 40, -(1 << 32) + 1):  # the C call would see their low 32 bits
        for name, call in (
                ("sinks", lambda: dsa.window_mla_decode(p, FAKE, FAKE, v, 4, FAKE, FAKE, FAKE, None, ws, 0)),
                ("window", lambda: dsa.window_mla_decode(p, FAKE, FAKE, 0, v, FAKE, FAKE, FAKE, None, ws, 0)),
                ("sinks", lambda: dsa.attention_mass(p, FAKE, FAKE, v, 4, FAKE, FAKE, lse, 0, mass, ws, 0)),
                ("window", lambda: dsa.attention_mass(p, FAKE, FAKE, 0, v, FAKE, FAKE, lse, 0, mass, ws, 0)),
                ("fresh", lambda: dsa.attention_mass(p, FAKE, FAKE, 0, 4, FAKE, FAKE, lse, v, mass, ws, 0)),
                ("sinks", lambda: dsa.tokens_evict(p, budgets, v, 0, mass, pools, FAKE, FAKE, FAKE, None, ws, 0)),
                ("recent", lambda: dsa.tokens_evict(p, budgets, 0, v, mass, pools, FAKE, FAKE, FAKE, None, ws, 0))):
            with pytest.raises(ValueError, match=name):
                call()
        with pytest.raises(ValueError, match="layers"):
            dsa.make_token_pools([(FAKE, 0, v, 0, 8448)])
    for name, bad in (("mass", z(2, 600, dtype=f32)), ("kept", z(2, 640, dtype=torch.int64)), ("kept", z(2, 641, dtype=i32)),
                      ("budgets", z(1, dtype=i32)), ("budgets", z(2, dtype=torch.int64))):
        a = {"mass": mass, "kept": None, "budgets": budgets, name: bad}
        with pytest.raises(ValueError, match=name):
            dsa.tokens_evict(p, a["budgets"], 0, 0, a["mass"], pools, FAKE, FAKE, FAKE, a["kept"], z(256, dtype=torch.uint8), 0)
