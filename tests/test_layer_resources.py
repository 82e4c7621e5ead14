"""What the layer's kernels take for granted of their code objects (no GPU needed)."""
from tests.test_kernel_resources import _kernels


def test_the_layers_table_begins_lds(tmp_path):
    # NF4's lookups take a byte of codes and a lane as an address in LDS: the table stands at 0, which it
    # does as long as the kernels have no static LDS in front of their dynamic LDS
    layer = {n: f for n, f in _kernels(tmp_path).items() if "k_layer_" in n}
    assert {part for part in ("k_layer_up", "k_layer_down") if any(part in n for n in layer)} == {"k_layer_up", "k_layer_down"}
    held = {n: f for n, f in layer.items() if f["group_segment_fixed_size"]}
    assert not held, held
