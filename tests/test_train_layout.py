"""The packed descriptors of the binding against the Structures of the C ABI."""
import pytest

from lora_rank_adapter_amd import _lib


@pytest.mark.parametrize("pack,struct", [(_lib.pack_mat, _lib.LoraMat), (_lib.pack_policy, _lib.LoraPolicy),
                                         (_lib.pack_hyper, _lib.LoraAdamwHyper)])
def test_packed_descriptors_have_the_structures_layout(pack, struct):
    values = list(range(1, len(struct._fields_) + 1))
    got = struct.from_buffer_copy(pack(*values))  # refuses fewer bytes than the structure has
    assert len(pack(*values)) == len(bytes(got))
    assert [getattr(got, name) for name, *_ in struct._fields_] == values
