"""The bounded cache's binding: arrays of other types or sizes, or with gaps, are refused by name before the library sees them."""
import pytest
import torch

import dsa_sparse_mla_paged_gb300 as dsa

FAKE = 0x10000  # never dereferenced
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _params():
    return dsa.make_params(batch=2, n_q=2, max_pages_per_req=10, num_pages=20, key_page_stride=8448, lat_page_stride=36864)


def z(*s, dtype=BF):
    return torch.zeros(s, dtype=dtype)


def window(**a):
    dsa.window_mla_decode(_params(), a["q"], FAKE, 4, 100, a["block_table"], a["ctx_lens"], a["out"], a["lse"], a["ws"], 0)


def mass(**a):
    dsa.attention_mass(_params(), a["q"], FAKE, 4, 100, a["block_table"], a["ctx_lens"], a["lse"], 2, a["mass"], a["ws"], 0)


def evict(**a):
    dsa.tokens_evict(_params(), a["budgets"], 4, 8, a["mass"], dsa.make_token_pools([]), a["block_table"], a["ctx_lens"], a["page_refs"],
                     a["kept"], a["ws"], 0)


def front(**a):
    dsa.latent_frontend(_params(), z(4, 96, 512), z(4, 96, 64), None, z(4, 512), z(4, 64), z(512), z(32, dtype=F32), None, FAKE,
                        a["block_table"], a["ctx_lens"], z(4, 96, 576), a["ws"], stream=0)


def good():
    return dict(q=z(4, 96, 576), out=z(4, 96, 512), lse=z(4, 96, dtype=F32), mass=z(2, 640, dtype=F32), kept=z(2, 640, dtype=I32),
                budgets=z(2, dtype=I32), block_table=z(2, 10, dtype=I32), ctx_lens=z(2, dtype=I32), page_refs=z(20, dtype=I32),
                ws=z(128, dtype=torch.uint8))


BAD = {
    "q": [z(4, 96, 576, dtype=torch.float16), z(4, 96, 576, dtype=F32), z(3, 96, 576), z(4, 96, 640)[:, :, :576],
          z(96, 4, 576).transpose(0, 1), z(1, 96, 576).expand(4, 96, 576)],
    "out": [z(4, 96, 512, dtype=torch.float16), z(4, 96, 512, dtype=F32), z(3, 96, 512), z(4, 96, 576)[:, :, :512]],
    "lse": [z(4, 96), z(4, 96, dtype=torch.float64), z(3, 96, dtype=F32), z(4, 192, dtype=F32)[:, ::2]],
    "block_table": [z(2, 10, dtype=torch.int64), z(2, 9, dtype=I32), z(2, 16, dtype=I32)[:, :10], z(1, 10, dtype=I32).expand(2, 10)],
    "ctx_lens": [z(2, dtype=torch.int64), z(1, dtype=I32), z(4, dtype=I32)[::2], z(1, dtype=I32).expand(2)],
    "page_refs": [z(20, dtype=torch.int64), z(19, dtype=I32), z(40, dtype=I32)[::2]],
}
CALLS = {window: ("q", "out", "lse", "block_table", "ctx_lens"), mass: ("q", "lse", "block_table", "ctx_lens"),
         evict: ("block_table", "ctx_lens", "page_refs"), front: ("block_table", "ctx_lens")}


@pytest.mark.parametrize("call", CALLS)
def test_good_arrays_addresses_and_larger_arrays_pass(lib, call):
    """(The workspace is too small, or not aligned: the library's own refusal.)"""
    for change in ({}, {k: FAKE for k in CALLS[call]}, dict(block_table=z(3, 10, dtype=I32), ctx_lens=z(5, dtype=I32))):
        with pytest.raises(dsa.DSAError) as e:
            call(**{**good(), **change})
        assert e.value.status in (dsa.DSA_ERR_WORKSPACE, dsa.DSA_ERR_INVALID)


@pytest.mark.parametrize("call,name,i", [(c, n, i) for c, names in CALLS.items() for n in names for i in range(len(BAD[n]))])
def test_other_arrays_are_refused(lib, call, name, i):
    with pytest.raises(ValueError, match=name):
        call(**{**good(), name: BAD[name][i]})


def test_what_may_be_left_out(lib):
    with pytest.raises(dsa.DSAError):  # no lse wanted
        window(**{**good(), "lse": None})
    for call, name in ((window, "out"), (mass, "lse"), (evict, "page_refs"), (front, "ctx_lens")):
        with pytest.raises(dsa.DSAError) as e:
            call(**{**good(), name: None})
        assert e.value.status == dsa.DSA_ERR_INVALID
