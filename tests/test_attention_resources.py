"""The kernels of the cache and of attention are in the built library, in every form that
their rules choose from, and none uses scratch memory or spills (CPU only): the waits of
the prompt kernel count loads, and a spill would be one more."""

import pytest

from test_build_resources import kernel_metadata, pytestmark  # noqa: F401

FAMILIES = {
    "append_kv_kernel": 2 * 2 * 2 * 2,      # types, head sizes, caches, heads per thread
    "decode_kernel": 2 * 2 * 2,
    "decode_join_kernel": 2 * 2 * 2,        # a group of threads a row, or all of them
    "prompt_kernel": 2 * 2 * 2 * 2,         # one or two halves of waves
    "prompt_join_kernel": 2 * 2 * 2,
}


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    return kernel_metadata(tmp_path_factory.mktemp("co"))


@pytest.mark.parametrize("family", FAMILIES)
def test_attention_kernels_do_not_spill(kernels, family):
    # mangled: the length of the name comes before it (fp8_decode_kernel is another)
    mine = {k: v for k, v in kernels.items() if f"{len(family)}{family}I" in k}
    assert len(mine) == FAMILIES[family], sorted(mine)
    for k, v in mine.items():
        assert v["private_segment_fixed_size"] == v["vgpr_spill_count"] == 0, k
        assert v["sgpr_spill_count"] == 0, k
