"""include/dg.h says of every call around the products that uses the workspace
that it does: two such calls on two streams need workspaces of their own.  No GPU."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
USERS = ["dg_m_grouped_layout_contiguous", "dg_m_grouped_layout_masked", "dg_m_grouped_scatter_fp8_contiguous",
         "dg_m_grouped_scatter_fp8_masked", "dg_lora_bf16_nt"]
OTHERS = ["dg_route_topk", "dg_route_topk_backward", "dg_k_grouped_scatter_fp8", "dg_m_grouped_gather",
          "dg_m_grouped_gather_weight_grad", "dg_m_grouped_rows_bound"]


def read(*path):
    with open(os.path.join(ROOT, *path)) as f:
        return f.read()


def comment_of(header, name):
    """The comment before a declaration; declarations that share one stand directly below one another."""
    at = re.search(rf"^int {name}\(", header, re.M).start()
    comment = header.rindex("/*", 0, at)
    return " ".join(header[comment:at].replace(" * ", " ").split())


def body_of(source, name):
    at = re.search(rf'extern "C" int {name}\(', source).start()
    return source[at:source.index("\n}", at)]


@pytest.mark.parametrize("name", USERS + OTHERS)
def test_the_header_names_the_calls_that_use_the_workspace(name):
    said = "Scratch: workspace" in comment_of(read("include", "dg.h"), name)
    assert said == (name in USERS), name


def test_the_list_above_is_the_code_s():
    csrc = ("moe_grouped_gemm_nt_amd", "csrc")
    source = "\n".join(read(*csrc, f) for f in ("route.hip", "expert_rows.hip", "lora.hip"))
    through = ["call_scratch", "run_layout", "scatter"]          # what reaches the workspace
    for name in USERS + OTHERS:
        uses = any(re.search(rf"(?<!\w){f}\(", body_of(source, name)) for f in through)
        assert uses == (name in USERS), name


def test_the_binding_of_a_workspace_speaks_of_them():
    text = comment_of(read("include", "dg.h"), "dg_bind_stream_workspace")
    assert "around the products" in text
