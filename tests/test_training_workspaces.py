"""Sizes of the workspaces of a training step's operators: what a call's path uses, and
no more (no GPU needed)."""
import pytest

import precision_collective_reduction_gb300 as pcr
from precision_collective_reduction_gb300 import build as lib_build


@pytest.fixture(scope="module")
def L():
    lib_build.build()
    return pcr.lib()


@pytest.mark.parametrize("T,V,H", [(513, 1000, 1), (4000, 100, 64), (16384, 32000, 8),
                                   (65536, 1000, 1), (65536, 1 << 20, 3)])
def test_embedding_gradient_sorted_in_one_cluster(L, T, V, H):
    # the sorted keys and tokens once, a bit for each row, and two partial rows for every
    # 8 tokens at the most; five parts, each rounded up to 256 bytes
    need = L.token_embed_backward_workspace_bytes(T, V, H)
    most = 2 * 4 * T + V // 8 + 2 * 4 * H * -(-T // 8) + 5 * 256
    least = 2 * 4 * T + V // 8
    assert least <= need <= most


@pytest.mark.parametrize("T", [65537, 70001, 1 << 20])
def test_embedding_gradient_sorted_through_memory(L, T):
    # keys and tokens twice, and up to 128 chunks' counts of 512 digits; one partial row
    # for every 32 tokens or more
    need = L.token_embed_backward_workspace_bytes(T, 1000, 1)
    assert 4 * 4 * T <= need <= 4 * 4 * T + 128 * 512 * 4 + 2 * 4 * -(-T // 16) + 9 * 256


def test_embedding_gradient_of_few_tokens_needs_none(L):
    assert L.token_embed_backward_workspace_bytes(512, 1 << 20, 8192) == 0
