"""C entry points refuse outputs and workspaces that share bytes with an
operand, before anything is launched (addresses are never dereferenced)."""
import pytest

A = 1 << 20  # an address, and room between operands
FAR = 1 << 30


def _embed(L, w=A, tok=FAR, out=2 * FAR, V=10, h=8, N=4, ld_w=8, ld_out=8):
    return L.lp_embedding(w, 0, V, h, ld_w, tok, N, 1.0, out, ld_out, None)


@pytest.mark.parametrize("kw", [
    dict(out=A), dict(out=A + 158), dict(out=A - 62), dict(out=A + 16, ld_out=16), dict(tok=2 * FAR),
    dict(tok=2 * FAR + 56), dict(tok=2 * FAR - 24), dict(w=A, out=A + 14, ld_w=16, ld_out=16),
    dict(out=A + 8, ld_w=8, ld_out=9)])
def test_embedding(lib_handle, kw):
    assert _embed(lib_handle, **kw) == 1 and b"overlaps" in lib_handle.lp_last_error()


@pytest.mark.parametrize("kw", [
    dict(dw=A), dict(dw=A + 60), dict(dw=A - 316), dict(tok=3 * FAR), dict(tok=3 * FAR + 312), dict(ws=3 * FAR),
    dict(ws=3 * FAR + 256), dict(ws=A), dict(tok=FAR, ws=FAR), dict(dw=2 * FAR)])
def test_embedding_backward(lib_handle, kw):
    L = lib_handle
    d = dict(g=A, tok=FAR, ws=2 * FAR, dw=3 * FAR)
    d.update(kw)
    need = L.lp_embedding_workspace_bytes(4, 8, 10)
    assert L.lp_embedding_backward(d["g"], 0, 4, 8, 8, d["tok"], 10, 1.0, 0, d["dw"], d["ws"], need, None) == 1
    assert b"overlaps" in L.lp_last_error()


@pytest.mark.parametrize("kw", [dict(p=A), dict(p=A + 1264), dict(s=A), dict(s=2 * FAR), dict(s=2 * FAR + 318),
                                dict(s=2 * FAR - 38)])
def test_quantize(lib_handle, kw):
    d = dict(w=A, p=2 * FAR, s=3 * FAR)
    d.update(kw)
    L = lib_handle
    assert L.lp_lm_head_w4_quantize(d["w"], 0, 10, 64, 64, 32, d["p"], 32, d["s"], 2, None) == 1
    assert b"overlap" in L.lp_last_error()


@pytest.mark.parametrize("kw", [dict(out=A), dict(out=A + 380), dict(out=2 * FAR), dict(out=2 * FAR + 316),
                                dict(out=3 * FAR), dict(out=3 * FAR - 116)])
def test_logits(lib_handle, kw):
    d = dict(x=A, p=2 * FAR, s=3 * FAR, out=4 * FAR)
    d.update(kw)
    L = lib_handle
    assert L.lp_lm_head_w4_logits(d["x"], 0, 3, 64, 64, d["p"], 32, d["s"], 2, 10, 32, d["out"], 2, 10, None) == 1
    assert b"overlaps" in L.lp_last_error()


@pytest.mark.parametrize("off,ld,ld_out", [(16, 16, 16), (15, 32, 32), (17, 32, 32), (31, 40, 40), (48, 32, 40),
                                           (32 * 3 + 15, 32, 32), (-15, 32, 32), (-17, 32, 32)])
def test_rules_outputs(lib_handle, off, ld, ld_out):
    """4 rows of 16 bf16 columns, the output `off` columns behind the logits."""
    L = lib_handle
    h = (A, 0, 4, 16, ld, None)
    assert L.lp_process_logits(*h, None, A + 2 * off, ld_out, None) == 1
    assert L.lp_processed_logprobs_entropy_backward(*h, FAR, None, 1.0, FAR, None, FAR, None, A + 2 * off, ld_out,
                                                    None) == 1
