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


def test_one_workspace_serves_every_window_and_layout():
    # The kernel's shape follows the window and the layouts; the bytes a call
    # dfc_paged_attention_workspace gives are a matter of the sizes alone
    import ctypes
    import lossless_entropy_coded_dfc_amd as dfc
    paged = pytest.importorskip("lossless_entropy_coded_dfc_amd.paged")
    lib = paged._lib()

    def args(window, v_stride, dim, heads, n, tokens, width, hint):
        kv = 8
        return paged.ATTENTION_ARGS.pack(256, 256, 16 * kv * dim, kv * dim, dim, *v_stride, 4096, 16, kv, dim, 0, heads,
                                         n, width, hint, tokens, 256, 256, heads * dim, dim, heads * dim, dim, 0, 256,
                                         width, 256, 256, 1.0, 1, window, 256, 0, 0)

    def need(a):
        out = ctypes.c_uint64()
        assert lib.dfc_paged_attention_workspace(a, ctypes.byref(out)) == 0
        return out.value

    for dim, heads, n, tokens, width, hint in [(128, 32, 1, 2048, 128, 0), (128, 32, 1, 513, 2032, 513),
                                               (64, 32, 4, 1900, 400, 1900), (128, 32, 16, 680, 2048, 333),
                                               (256, 16, 2, 700, 1000, 0), (80, 8, 3, 300, 9, 0), (128, 32, 64, 64, 512, 1)]:
        sizes = dim, heads, n, tokens, width, hint
        plain = 16 * 8 * dim, 8 * dim, dim
        most = need(args(0, plain, *sizes))
        for window in (0, 1, 64, 777, 5000):
            for layout in (plain, (16 * 8 * dim, dim, 16 * dim)):
                a = args(window, layout, *sizes)
                assert need(a) == most, (sizes, window, layout)
                # no bytes given: refused before anything is launched
                assert lib.dfc_paged_attention(a, None) == dfc.ESIZE, (sizes, window, layout)
