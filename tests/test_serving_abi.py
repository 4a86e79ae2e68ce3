"""Host validation of the calls around the decode step (CPU: every case is
rejected before any CUDA call) and the binding's own checks."""
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
    need = dsa.workspace_size(p)
    args = {**args, "ws": FAKE, "bytes": need, **change}
    return getattr(dsa.load(), fn)(ctypes.byref(p), *args.values(), None)


PREFIX = dict(q=FAKE, lat=FAKE, pages=FAKE, prefix=128, table=FAKE, ctx=FAKE, out=FAKE, lse=None)


@pytest.mark.parametrize("change", [
    dict(q=None), dict(q=FAKE + 2), dict(lat=FAKE + 8), dict(lat=None), dict(pages=None), dict(prefix=-64), dict(prefix=100),
    dict(prefix=640), dict(table=None), dict(ctx=None), dict(out=None), dict(out=FAKE + 4), dict(ws=None), dict(ws=FAKE + 4)])
def test_prefix_attention_rejects(lib, change):
    assert _call("dsa_prefix_mla_decode", _params(), PREFIX, **change) == INVALID


def test_prefix_attention_workspace(lib):
    p = _params()
    assert _call("dsa_prefix_mla_decode", p, PREFIX, bytes=dsa.workspace_size(p) - 1) == WORKSPACE
    # no prefix needs no page list; one that leaves no room for the new tokens is refused
    assert _call("dsa_prefix_mla_decode", p, PREFIX, pages=None, prefix=0, bytes=0) == WORKSPACE
    assert _call("dsa_prefix_mla_decode", p, PREFIX, prefix=576, bytes=0) == WORKSPACE
    assert _call("dsa_prefix_mla_decode", _params(n_q=65), PREFIX, prefix=576, bytes=0) == INVALID


def _pools(*pools):
    return dsa.make_pools(pools)


RESIZE = dict(new=FAKE, pools=None, n=0, table=FAKE, ctx=FAKE, refs=FAKE)
COMPACT = dict(pools=None, n=0, table=FAKE, ctx=FAKE, refs=FAKE, map=None, live=None)
FORK = dict(n=2, src=FAKE, dst=FAKE, table=FAKE, ctx=FAKE, refs=FAKE)


@pytest.mark.parametrize("fn,args", [("dsa_pages_resize", RESIZE), ("dsa_pages_compact", COMPACT)])
def test_page_operations_reject(lib, fn, args):
    p = _params()
    for name in ("table", "ctx", "refs"):
        assert _call(fn, p, args, **{name: None}) == INVALID
    assert _call(fn, p, args, n=-1) == INVALID
    assert _call(fn, p, args, n=1) == INVALID
    good = (FAKE, 64, 64)
    for bad in ((None, 64, 64), (FAKE + 8, 64, 64), (FAKE, 8, 64), (FAKE, 40, 64), (FAKE, 64, 48), (FAKE, 64, 72)):
        pools, n = _pools(good, bad)
        assert _call(fn, p, args, pools=pools, n=n) == INVALID, bad
    pools, n = _pools(*[good] * 65)
    assert _call(fn, p, args, pools=pools, n=n) == UNSUPPORTED
    pools, n = _pools((FAKE, (1 << 32) + 16, 1 << 33))
    assert _call(fn, p, args, pools=pools, n=n) == UNSUPPORTED
    pools, n = _pools(*[good] * 64)
    assert _call(fn, p, args, pools=pools, n=n, bytes=0) == WORKSPACE
    assert _call(fn, p, args, ws=None) == INVALID


def test_resize_and_fork_reject(lib):
    p = _params()
    assert _call("dsa_pages_resize", p, RESIZE, new=None) == INVALID
    for change in (dict(n=-1), dict(n=3), dict(src=None), dict(dst=None), dict(table=None), dict(ctx=None),
                   dict(refs=None)):
        assert _call("dsa_pages_fork", p, FORK, **change) == INVALID, change
    assert _call("dsa_pages_fork", p, FORK, bytes=0) == WORKSPACE
    assert _call("dsa_pages_fork", p, FORK, n=0, src=None, dst=None) == dsa.DSA_OK  # nothing to launch


VERIFY = dict(vocab=100, dtype=0, p=FAKE, ps=100, q=FAKE, qs=100, tokens=FAKE, counts=None, u=FAKE, ctx=FAKE, acc=FAKE, out=FAKE,
              new=FAKE)


@pytest.mark.parametrize("change", [
    dict(vocab=0), dict(vocab=-1), dict(dtype=3), dict(dtype=-1), dict(p=None), dict(p=FAKE + 2), dict(ps=99), dict(q=FAKE + 1),
    dict(qs=99), dict(dtype=1, p=FAKE + 1), dict(tokens=None), dict(u=None), dict(acc=None), dict(out=None), dict(ctx=None)])
def test_verify_rejects(lib, change):
    assert _call("dsa_verify_draft", _params(), VERIFY, **change) == INVALID


def test_verify_limits(lib):
    p = _params()
    assert _call("dsa_verify_draft", p, VERIFY, vocab=(1 << 24) + 1, ps=1 << 25, qs=1 << 25) == UNSUPPORTED
    assert _call("dsa_verify_draft", p, VERIFY, bytes=0) == WORKSPACE
    assert _call("dsa_verify_draft", p, VERIFY, dtype=2, p=FAKE + 2, q=None, qs=0, bytes=0) == WORKSPACE
    assert _call("dsa_verify_draft", p, VERIFY, ctx=None, new=None, bytes=0) == WORKSPACE
    assert _call("dsa_verify_draft", _params(n_q=1), VERIFY, tokens=None, bytes=0) == WORKSPACE


def test_null_params_and_bad_params(lib):
    for fn, args in (("dsa_prefix_mla_decode", PREFIX), ("dsa_pages_resize", RESIZE), ("dsa_pages_fork", FORK),
                     ("dsa_pages_compact", COMPACT), ("dsa_verify_draft", VERIFY)):
        f = getattr(lib, fn)
        assert f(None, *args.values(), FAKE, 0, None) == INVALID, fn
        p = _params()
        p.batch = 0
        assert f(ctypes.byref(p), *args.values(), FAKE, 0, None) == INVALID, fn
        p = _params()
        p.page_size = 32
        assert f(ctypes.byref(p), *args.values(), FAKE, 0, None) == UNSUPPORTED, fn


def test_binding_checks():
    import torch

    p = _params()
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="length"):
        dsa.pages_fork(p, i, i[:1], None, None, None, i)
    t = torch.zeros(2, 2, 8)

    def call(target, draft):
        dsa.verify_draft(p, target, draft, i, None, i, None, i, i, None, i)

    for target, draft in ((t.double(), None), (t[:1], None), (t.transpose(1, 2), None), (t[:, :, ::2], None), (t, t),
                          (t, t[:, :1].to(torch.bfloat16)), (t, t[:, :1, :4].contiguous()),
                          (torch.zeros(2, 3, 8)[:, :2], None)):
        with pytest.raises(ValueError, match="verify_draft"):
            call(target, draft)


@pytest.mark.parametrize("n_q", [1, 3])
def test_binding_refuses_rows_that_share_elements(n_q):
    """Expanded and overlapping rows: the kernel would read past the storage's end."""
    import torch

    p = _params(batch=4, n_q=n_q)
    i = torch.zeros(4 * n_q, dtype=torch.int32)
    u = torch.zeros(4, n_q)
    good_t, good_d = torch.rand(4, n_q, 50), torch.rand(4, max(n_q - 1, 1), 50) if n_q > 1 else None

    def call(target, draft):
        dsa.verify_draft(p, target, draft, i[:4 * (n_q - 1)].view(4, n_q - 1), None, u, None, i[:4], i.view(4, n_q), None, i)

    one, line = torch.rand(50), torch.rand(800)
    cases = [one.expand(4, n_q, 50), one.expand(4 * n_q, 50), torch.rand(4, 1, 50).expand(4, max(n_q, 2), 50)[:, :n_q]
             if n_q > 1 else torch.rand(1, 1, 50).expand(4, 1, 50), torch.rand(1, n_q, 50).expand(4, n_q, 50),
             line.as_strided((4, n_q, 50), (7 * n_q, 7, 1)), line.as_strided((4 * n_q, 50), (49, 1)),
             torch.rand(2, 2, n_q, 50).transpose(0, 1)]
    for bad in cases:
        with pytest.raises(ValueError, match="verify_draft"):
            call(bad, good_d)
        if n_q > 1:
            with pytest.raises(ValueError, match="verify_draft"):
                call(good_t, bad[..., :n_q - 1, :] if bad.dim() >= 3 else bad[:4 * (n_q - 1)])


def test_binding_takes_one_row_of_any_stride():
    """A single row has no distance to the next: the stride passed on is at least the vocabulary."""
    import torch

    for t in (torch.rand(50), torch.rand(1, 50), torch.rand(1, 1, 50), torch.rand(50).expand(1, 1, 50),
              torch.rand(3, 50)[::2][:1], torch.rand(400).as_strided((1, 1, 50), (3, 7, 1))):
        assert dsa._prob_rows("target", t, 1)[1] >= 50
    assert dsa._prob_rows("target", torch.rand(4, 2, 60)[:, :, 5:55], 8)[1] == 60
    assert dsa._prob_rows("target", torch.rand(4, 3, 60)[:, 1:2], 4)[1] == 180
    assert dsa._prob_rows("target", torch.rand(2, 2, 3, 60), 12)[1] == 60


def test_binding_refuses_arrays_of_other_types_and_sizes():
    """int64 tokens, one row of numbers for the whole batch, slices of wider arrays."""
    import torch

    p = _params(batch=4, n_q=3)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    good = dict(tokens=i(4, 2), counts=i(4), u=torch.zeros(4, 3), ctx=i(4))

    def verify(**change):
        a = {**good, **change}
        dsa.verify_draft(p, torch.rand(4, 3, 9), torch.rand(4, 2, 9), a["tokens"], a["counts"], a["u"], a["ctx"], i(4), i(4, 3),
                         i(4), i(1))

    for name, bad in (("tokens", i(4, 2).long()), ("tokens", i(1, 2).expand(4, 2)), ("tokens", i(4, 3)[:, :2]),
                      ("tokens", i(3, 2)), ("counts", i(4).long()), ("counts", i(1).expand(4)), ("counts", i(3)),
                      ("u", torch.zeros(1, 3).expand(4, 3)), ("u", torch.zeros(4, 3).double()), ("u", torch.zeros(4, 2)),
                      ("u", torch.zeros(3, 4).t()), ("ctx", i(4).float()), ("ctx", i(8)[::2])):
        with pytest.raises(ValueError, match="verify_draft: "):
            verify(**{name: bad})
    for src, dst in ((i(2).long(), i(2)), (i(2), i(1).expand(2)), (i(4)[::2], i(2))):
        with pytest.raises(ValueError, match="pages_fork: "):
            dsa.pages_fork(p, src, dst, None, None, None, i(1))
    for new in (i(4).long(), i(3), i(1).expand(4)):
        with pytest.raises(ValueError, match="pages_resize: "):
            dsa.pages_resize(p, new, dsa.make_pools([]), None, None, None, i(1))


def test_page_operations_limit_the_number_of_pages(lib):
    """Their page loops count in 32 bits."""
    for n, status in ((1 << 30, WORKSPACE), ((1 << 30) + 1, UNSUPPORTED), (2 ** 31 - 1, UNSUPPORTED)):
        p = _params(num_pages=n)
        for fn, args in (("dsa_pages_resize", RESIZE), ("dsa_pages_compact", COMPACT), ("dsa_pages_fork", FORK)):
            assert _call(fn, p, args, bytes=0) == status, (fn, n)


def _size(batch, n_q, topk, max_pages, num_pages=1000):
    return dsa.workspace_size(_params(batch=batch, n_q=n_q, topk=topk, max_pages_per_req=max_pages, num_pages=num_pages))


@pytest.mark.parametrize("case,size", [  # what the decode step's own regions come to
    ((8, 1, 2048, 1024), 31335424), ((64, 1, 2048, 1024), 250561536), ((12, 6, 2048, 700), 272677632),
    ((1, 2048, 2048, 2344), 9083921152), ((256, 8, 2048, 1600), 8482808576)])
def test_serving_scratch_shares_the_decode_steps_workspace(lib, case, size):
    assert _size(*case) == size
    assert _size(*case, num_pages=50000) == size  # the page lists too


def test_workspace_of_few_rows(lib):
    """The prefix attention's partials of 76 CTA pairs do not fit in a few rows' room: 21 MB more."""
    for case, own in (((1, 1, 2048, 64), 3554304), ((2, 1, 2048, 10), 7047680), ((64, 1, 128, 1024), 45229056)):
        rows = case[0] * case[1]
        assert own < _size(*case) <= own + rows * 0.6e6 + 21e6


def test_verification_takes_a_workspace_of_its_error_word(lib):
    p = _params(batch=256, n_q=8, max_pages_per_req=1600)
    assert _call("dsa_verify_draft", p, VERIFY, bytes=255) == WORKSPACE
    assert _call("dsa_verify_draft", p, VERIFY, bytes=256, ws=FAKE + 8) == INVALID
    assert _call("dsa_verify_draft", p, VERIFY, bytes=256, ws=None) == INVALID


def test_binding_refuses_page_lists_of_other_types_and_sizes():
    import torch

    p = _params()
    for pages in (torch.zeros(2, dtype=torch.int64), torch.zeros(1, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError, match="prefix_mla_decode: prefix_pages"):
            dsa.prefix_mla_decode(p, FAKE, FAKE, pages, 128, FAKE, FAKE, FAKE, None, torch.zeros(1))
