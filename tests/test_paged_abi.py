"""The paged cache's argument structures as the Python binding packs them
against the C compiler's layout of include/dfc.h, field by field."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FIELDS = {
    "dfc_paged_cache": ("CACHE", ["k_dev", "v_dev", "k_stride", "v_stride", "n_pages", "page_size", "kv_heads",
                                  "head_dim", "dtype"]),
    "dfc_plan_args": ("PLAN_ARGS", ["n_requests", "max_pages", "page_size", "n_ring", "tokens", "context_lens",
                                    "new_lens", "block_table", "table_stride", "free_pages", "cursor", "seq_lens",
                                    "cu_q", "slots", "positions", "cursor_out", "status_dev"]),
    "dfc_append_args": ("APPEND_ARGS", ["cache", "tokens", "k_dev", "v_dev", "k_src_stride", "v_src_stride", "slots",
                                        "source_dtype", "q_heads", "q_dev", "q_out_dev", "q_stride", "q_out_stride",
                                        "rot_dim", "interleaved", "max_positions", "positions", "rotary_dev",
                                        "status_dev"]),
    "dfc_attention_args": ("ATTENTION_ARGS", ["cache", "heads", "n_requests", "max_pages", "max_q_len", "tokens",
                                              "q_dev", "out_dev", "q_stride", "out_stride", "lse_dev", "block_table",
                                              "table_stride", "cu_q", "seq_lens", "scale", "causal", "window",
                                              "workspace_dev", "workspace_bytes", "status_dev"]),
}
ARRAYS = {"k_stride": 3, "v_stride": 3, "k_src_stride": 2, "v_src_stride": 2, "q_stride": 2, "q_out_stride": 2,
          "out_stride": 2, "cache": 13}


@pytest.mark.parametrize("name", sorted(FIELDS))
def test_layout(name, tmp_path):
    paged = pytest.importorskip("lossless_entropy_coded_dfc_amd.paged")
    packer, fields = FIELDS[name]
    packer = getattr(paged, packer)
    lines = "\n".join(f'printf("%zu %zu\\n", offsetof({name}, {f}), sizeof(x.{f}));' for f in fields)
    src = tmp_path / "layout.c"
    src.write_text(f"#include <stdio.h>\n#include \"dfc.h\"\n"
                   f"int main(void) {{ {name} x; (void)x; {lines}\n printf(\"%zu 0\\n\", sizeof(x)); return 0; }}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    rows = [tuple(map(int, line.split())) for line in
            subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()]
    assert packer.size == rows[-1][0]
    # one field at a time: its value lands at its offset and nowhere else
    values = len(packer.unpack(bytes(packer.size)))
    at = 0
    for field, (offset, size) in zip(fields, rows):
        for k in range(ARRAYS.get(field, 1)):
            mark = [0] * values
            mark[at] = 1
            data = packer.pack(*mark)
            places = [i for i, b in enumerate(data) if b]
            assert all(offset <= i < offset + size for i in places), field
            if field not in ("cache", "scale"):
                assert places == [offset + k * size // ARRAYS.get(field, 1)], field
            at += 1
    assert at == values
