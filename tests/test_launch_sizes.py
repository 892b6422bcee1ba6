"""Launches of 2^32 threads and more are refused before anything runs: the runtime would start a part of them and report
no error.  (Without a GPU: the sizes are far beyond any memory, and nothing is read.)"""
import ctypes
import os

import pytest

FAKE = ctypes.c_void_p(0x1000)          # never dereferenced


@pytest.fixture(scope="module")
def lib():
    import w4_dequant_gemm_amd as w4
    if not os.path.exists(w4.library_path):
        from w4_dequant_gemm_amd import build
        build.build()
    return w4.lib()


def test_launches_beyond_32_bits_are_refused(lib):
    import w4_dequant_gemm_amd as w4
    one = (ctypes.c_float * 1)(1.0)
    most = 1 << 40

    def refused(status):
        assert status == 3 and "invalid configuration" in w4.w4_last_error(), w4.w4_last_error()

    # 2^32 words of codes, groups, rows of one group, NF4 blocks
    refused(lib.w4_prepack(FAKE, FAKE, FAKE, 1 << 27, 256, 128, 1, FAKE, FAKE, None))
    refused(lib.w4_quantize_blockwise(FAKE, 1 << 31, 256, 128, 1, one, 1, FAKE, FAKE, FAKE, None, None))
    refused(lib.w4_quantize_blockwise(FAKE, 1 << 22, 1024, 1024, 1, one, 1, FAKE, FAKE, FAKE, None, None))
    refused(lib.w4_nf4_quantize(FAKE, 1 << 30, 256, FAKE, FAKE, FAKE, None))
    # products: workgroups of one or two rows by 16 columns, of tiles
    refused(lib.w4a16_gemm(FAKE, 1, 4096, FAKE, FAKE, most, 128, FAKE, None, 0, None))
    refused(lib.w4a16_gemm(FAKE, most, 96, FAKE, FAKE, 8, 32, FAKE, None, 0, None))
    refused(lib.w4a16_gemm(FAKE, most, 512, FAKE, FAKE, 8, 32, FAKE, FAKE, 1 << 62, None))
    refused(lib.w4a16_gemm(FAKE, most, 512, FAKE, FAKE, 4096, 32, FAKE, FAKE, 1 << 62, None))


def test_attention_over_more_tiles_than_a_launch_has(lib):
    """65535 sequences planned for chunks of 4096 tokens: a workgroup for each 64 rows of each head."""
    import w4_dequant_gemm_amd as w4
    from test_decode_abi import _attend, _cache
    status = _attend(lib, _cache(kv_heads=64), T=65535 + 4096, hq=64, qs=64 * 128, B=65535, max_q=4096, max_kv=4096, pages=4096, tree=None,
                     words=0, ws=FAKE, ws_bytes=1 << 60)
    assert status == 3 and "invalid configuration" in w4.w4_last_error(), w4.w4_last_error()
