"""The structs of include/wush.h as a C compiler lays them out are what the binding packs."""
import os
import shutil
import struct
import subprocess

import pytest

aq = pytest.importorskip("activation_quantization_b200")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FIELDS = {
    "wush_norm_spec": (aq._NORM_SPEC, "kind dtype weight bias weight_offset eps"),
    "wush_residual_norm_args": (
        aq._RESIDUAL_NORM_ARGS,
        "y gate r r_out h y_stride gate_stride r_stride r_out_stride h_stride rows d post.kind post.dtype post.weight "
        "post.bias post.weight_offset post.eps pre.kind pre.dtype pre.weight pre.bias pre.weight_offset pre.eps "
        "y_dtype gate_dtype r_dtype h_dtype gate_act residual_scale branch_scale"),
    "wush_lora_args": (
        aq._LORA_ARGS,
        "x adapter a b ranks scale y_in y workspace x_stride y_in_stride y_stride tokens d_in d_out n_adapters rank "
        "workspace_bytes dtype"),
}


def _offsets(fmt):
    """Offset of each value of a struct format in native alignment."""
    codes, n = [], ""
    for ch in fmt.format.lstrip("@"):
        if ch.isdigit():
            n += ch
        else:
            codes += [ch] * int(n or 1)
            n = ""
    out, prefix = [], "@"
    for ch in codes:
        prefix += ch
        out.append(struct.calcsize(prefix) - struct.calcsize("@" + ch))
    return out


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_field_offsets(tmp_path):
    lines = []
    for name, (_, fields) in FIELDS.items():
        lines += [f'printf("{name} {f} %zu\\n", offsetof({name}, {f}));' for f in fields.split()]
        lines.append(f'printf("{name} sizeof %zu\\n", sizeof({name}));')
    src = tmp_path / "o.c"
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"wush.h\"\nint main(void) {\n" + "\n".join(lines) +
                   "\nreturn 0; }\n")
    subprocess.run(["gcc", "-std=gnu99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "o")],
                   check=True)
    got = {}
    for line in subprocess.run([str(tmp_path / "o")], capture_output=True, text=True, check=True).stdout.splitlines():
        name, field, value = line.split()
        got[name, field] = int(value)
    for name, (fmt, fields) in FIELDS.items():
        fields = fields.split()
        offsets = _offsets(fmt)
        assert len(offsets) == len(fields), name
        for f, o in zip(fields, offsets):
            assert got[name, f] == o, (name, f)
        assert 0 <= got[name, "sizeof"] - fmt.size < 8              # at most the end's padding
