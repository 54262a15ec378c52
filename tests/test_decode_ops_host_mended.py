"""The operators between the GEMVs without a GPU, where they had gone wrong: empty calls, the build."""
import quant_dequant_gemv_q4_b200 as qg
from test_decode_ops_host import A, L, heads, norm_rope  # noqa: F401


def test_no_tokens_need_no_addresses(L):
    """T = 0 with a rotation: an empty array's address is null."""
    assert norm_rope(L, T=0, pos=None) == qg.QG_OK
    assert norm_rope(L, T=0, pos=None, q=heads(ptr=None), k=heads(ptr=None), qo=heads(ptr=None), ko=heads(ptr=None)) == qg.QG_OK
    assert norm_rope(L, T=0, pos=None, R=65) == qg.QG_ERR_SHAPE and norm_rope(L, T=0, pos=None, pairing=3) == qg.QG_ERR_VARIANT
    none = heads(ptr=None)
    assert L.qg_kv4_append(none, none, 0, 2, 128, None, 0.0, None, A, 64, 0, None, A, 4, 32, None) == qg.QG_OK
    assert L.qg_kv4_append(none, none, 0, 2, 128, None, 0.0, None, A, 64, 0, None, None, 0, 32, None) == qg.QG_OK
    assert L.qg_kv4_read(A, 4, 32, 2, 128, None, 0, none, none, None) == qg.QG_OK
    assert L.qg_attn_kv4(none, 0, 0, None, 0, 4, 2, 128, None, 0, 32, None, 0, None, 1.0, none, None, 0, None) == qg.QG_OK
    assert L.qg_sample(None, 0, 100, 100, 1, None, None, None, None, None, None, None, 0, None) == qg.QG_OK
