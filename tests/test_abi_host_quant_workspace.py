"""Workspace of the products of 8-bit rows, judged on the host: what one call's operands need is never more
than what any operands need, and holds no copy of operands that are read in place."""
import pytest

SPLIT = 128 << 20  # partial sums of a split product, at most


@pytest.fixture(scope="module")
def lib():
    from gmm_em_amd import ops

    return ops.lib


def test_sizes(lib):
    call = lib.gmm_quantized_product_call_workspace_bytes
    for n, d, v in ((0, 1, 1), (1, 768, 16384), (16, 131071, 1 << 22), (17, 1, 1), (17, 128, 1), (64, 768, 16384),
                    (128, 8192, 4096), (257, 400, 1025), (777, 1003, 5001), (2100, 130944, 40), (2100, 130999, 40),
                    (8192, 8192, 131072), (1 << 40, 1000, 100_000), (1 << 40, 131071, 1 << 22)):
        most = lib.gmm_quantized_product_workspace_bytes(n, d, v)
        dp = (d + 127) // 128 * 128
        for pq in (dp, dp + 16, dp + 1):
            for pw in (dp, dp + 16, dp + 1):
                for at in (4096, 4097):
                    need = call(at, n, d, pq, at, v, pw)
                    print(n, d, v, pq, pw, at, need, most)
                    assert 256 <= need <= most and need % 256 == 0
                    if d == dp and at == 4096:
                        in_place = (0 if pq % 16 == 0 else min(n * dp, 256 << 20)) + (0 if pw % 16 == 0 else v * dp)
                        assert need <= SPLIT + in_place + 768
    # a wide head's product with a batch: nothing to lay out, nothing split
    assert call(4096, 8192, 8192, 8192, 4096, 131072, 8192) == 256


def test_invalid_sizes(lib):
    call = lib.gmm_quantized_product_call_workspace_bytes
    for n, d, ldq, v, ldw in ((-1, 8, 8, 8, 8), (8, 0, 8, 8, 8), (8, 8, 8, 0, 8), (8, 1 << 17, 1 << 17, 8, 1 << 17),
                              (8, 8, 8, (1 << 22) + 1, 8), (8, 8, 7, 8, 8), (8, 8, 8, 8, 7), ((1 << 40) + 1, 8, 8, 8, 8)):
        assert call(4096, n, d, ldq, 4096, v, ldw) == 0
