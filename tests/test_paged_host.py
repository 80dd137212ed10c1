"""Host-side checks of the paged cache calls (no GPU needed): refusals come back before
any launch."""
import pytest
import torch

import exact_io_aware_54_b200 as fa
from exact_io_aware_54_b200 import build as fa_build

P = 0x10000  # a 16-byte aligned fake device address; validation fails before any use
ST = {v: k for k, v in fa.STATUS.items()}
INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = (ST["FA_ERR_" + n] for n in (
    "INVALID_ARG", "UNSUPPORTED", "ALIGNMENT", "WORKSPACE"))


@pytest.fixture(scope="module")
def lib():
    fa_build.build()
    return fa.load()


PAGES = [(dict(kp=None), INVALID), (dict(vp=None), INVALID), (dict(table=None), INVALID), (dict(ks=None), INVALID),
         (dict(vs=None), INVALID), (dict(B=0), INVALID), (dict(H=0), INVALID), (dict(np=0), INVALID),
         (dict(ps=0), INVALID), (dict(mp=-1), INVALID), (dict(np=1 << 20, ps=1 << 11), INVALID),
         (dict(mp=1 << 20, ps=1 << 11), INVALID), (dict(d=96), UNSUPPORTED), (dict(kp=P + 8), ALIGNMENT),
         (dict(vp=P + 8), ALIGNMENT), (dict(table=P + 2), ALIGNMENT), (dict(ws=None), WORKSPACE),
         (dict(ws=P + 8), WORKSPACE), (dict(wsb=8), WORKSPACE)]


def _defaults(kw):
    a = dict(k=P, v=P, q=P, rs=512, cu=P, table=P, lens=P, kp=P, vp=P, ks=P, vs=P, o=P, lse=P, B=2, H=4, Hq=4, total=8,
             np=16, ps=16, mp=4, maxq=8, maxk=64, d=128, ws=P, wsb=1 << 30)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,status", PAGES + [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(cu=None), INVALID), (dict(lens=None), INVALID),
    (dict(total=0), INVALID), (dict(rs=511), INVALID), (dict(rs=516), ALIGNMENT), (dict(k=P + 8), ALIGNMENT),
    (dict(v=P + 8), ALIGNMENT), (dict(cu=P + 2), ALIGNMENT), (dict(lens=P + 2), ALIGNMENT)])
def test_write_refusals(lib, kw, status):
    a = _defaults(kw)
    assert lib.fa_cache_write(a["k"], a["v"], a["rs"], a["rs"], a["cu"], a["table"], a["lens"], a["kp"], a["vp"],
                              a["ks"], a["vs"], a["B"], a["H"], a["total"], a["np"], a["ps"], a["mp"], a["d"],
                              a["ws"], a["wsb"], None) == status


@pytest.mark.parametrize("kw,status", PAGES + [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(cu=None), INVALID), (dict(total=0), INVALID),
    (dict(k=P + 8), ALIGNMENT), (dict(v=P + 8), ALIGNMENT), (dict(cu=P + 2), ALIGNMENT)])
def test_read_refusals(lib, kw, status):
    a = _defaults(kw)
    assert lib.fa_cache_read(a["kp"], a["vp"], a["ks"], a["vs"], a["cu"], a["table"], a["k"], a["v"], a["B"], a["H"],
                             a["total"], a["np"], a["ps"], a["mp"], a["d"], a["ws"], a["wsb"], None) == status


ATTEND = PAGES + [
    (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(lse=None), INVALID), (dict(lens=None), INVALID),
    (dict(Hq=6), INVALID), (dict(Hq=0), INVALID), (dict(maxk=65), INVALID), (dict(maxk=-1), INVALID),
    (dict(q=P + 8), ALIGNMENT), (dict(o=P + 8), ALIGNMENT), (dict(lse=P + 4), ALIGNMENT), (dict(lens=P + 2), ALIGNMENT),
    (dict(ks=P + 2), ALIGNMENT), (dict(vs=P + 1), ALIGNMENT)]


@pytest.mark.parametrize("kw,status", ATTEND + [
    (dict(cu=None), INVALID), (dict(total=0), INVALID), (dict(maxq=0), INVALID), (dict(rs=504), INVALID),
    (dict(rs=516), ALIGNMENT), (dict(cu=P + 2), ALIGNMENT), (dict(total=1 << 30), INVALID)])
def test_fwd_refusals(lib, kw, status):
    a = _defaults(kw)
    assert lib.fa_fwd_paged(a["q"], a["rs"], a["kp"], a["vp"], a["ks"], a["vs"], a["cu"], a["table"], a["lens"], a["o"],
                            a["lse"], a["B"], a["Hq"], a["H"], a["total"], a["np"], a["ps"], a["mp"], a["maxq"],
                            a["maxk"], a["d"], 1, 0.0, a["ws"], a["wsb"], None) == status


@pytest.mark.parametrize("kw,status", ATTEND + [(dict(ks=None, vs=None), INVALID)])
def test_decode_refusals(lib, kw, status):
    a = _defaults(kw)
    assert lib.fa_decode_paged_q8(a["q"], a["kp"], a["vp"], a["ks"], a["vs"], a["table"], a["lens"], a["B"], a["Hq"],
                                  a["H"], a["np"], a["ps"], a["mp"], a["maxk"], a["d"], 0.0, a["o"], a["lse"],
                                  a["ws"], a["wsb"], None) == status


def test_workspace_size(lib):
    assert fa.fa_paged_workspace_size(4, 32, 8, 512, 16384, 128) > 256
    for bad in ((0, 32, 8, 1, 1, 128), (1, 30, 8, 1, 1, 128), (1, 8, 8, 0, 1, 128), (1, 8, 8, 1, -1, 128),
                (1, 8, 8, 1, 1, 96), (1, 8, 8, 2 ** 31 - 1, 2 ** 31 - 1, 128)):
        assert fa.fa_paged_workspace_size(*bad) == 0


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    pages = torch.zeros(3, 16, 4, 64, dtype=torch.bfloat16)
    cu, table = torch.tensor([0, 2], dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32)
    lens = torch.tensor([2], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_cache_write(x, x, pages, pages, cu, table, lens)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_cache_read(pages, pages, cu, table, 2)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_fwd_paged(x, pages, pages, cu, table, lens, 2, 2)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_decode_paged_q8(x, pages, pages, pages, pages, table, lens, 2)
    with pytest.raises(ValueError, match="together"):
        fa._pages_of(pages, pages, pages, None, table, 1, 0)
