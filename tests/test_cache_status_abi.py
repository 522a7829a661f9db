"""The statuses of the workspace queries' refusals (no GPU needed): those of the calls that take the workspaces."""
import pytest
import torch

from test_cache_abi import hsp  # noqa: F401  (the module's fixture)

ATTENTION = [((0, 1, 576, 512, True), "INVALID_ARG"), ((16, 0, 576, 512, True), "INVALID_ARG"), ((-4, 2, 64, 64, False), "INVALID_ARG"),
             ((16, 3, 576, 512, True), "UNSUPPORTED_SHAPE"), ((16, 1, 96, 96, False), "UNSUPPORTED_SHAPE"),
             ((16, 1, 576, 512, False), "UNSUPPORTED_SHAPE"), ((16, 1, 576, -1, True), "UNSUPPORTED_SHAPE"),
             ((1 << 17, 1, 512, 512, True), "UNSUPPORTED_SHAPE"), ((16, 1, 576, 512 + 2 ** 32, True), "UNSUPPORTED_SHAPE"),
             ((16 - 2 ** 32, 1, 576, 512, True), "INVALID_ARG")]


@pytest.mark.parametrize("args,want", ATTENTION)
def test_attention_workspace(hsp, args, want):  # noqa: F811
    with pytest.raises(hsp.ProjError) as ei:
        hsp.paged_attention_workspace_bytes(*args)
    assert ei.value.status_name == "PROJ_ERR_" + want
    assert len(str(ei.value)) > len("PROJ_ERR_" + want) + 10


@pytest.mark.parametrize("shape,pages,n,want", [((4, 8), 32, -1, "INVALID_ARG"), ((0, 8), 32, 3, "UNSUPPORTED_SHAPE"),
                                                ((4, 0), 32, 3, "UNSUPPORTED_SHAPE"), ((4, 8), 0, 3, "UNSUPPORTED_SHAPE"),
                                                ((4, 8), -1, 3, "INVALID_ARG"), ((4, 8), (1 << 30) + 1, 0, "UNSUPPORTED_SHAPE"),
                                                ((4, 8), 32 - 2 ** 32, 3, "INVALID_ARG"), ((4, 8), 32, 3 - 2 ** 32, "INVALID_ARG")])
def test_cache_workspace(hsp, shape, pages, n, want):  # noqa: F811
    with pytest.raises(hsp.ProjError) as ei:
        hsp.cache_workspace_bytes(torch.zeros(shape, dtype=torch.int32), pages, n)
    assert ei.value.status_name == "PROJ_ERR_" + want
