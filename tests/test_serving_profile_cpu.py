"""profiles/serving_operators.md was captured from the serving kernels as they are: it carries a digest of their sources
without comments and white space, and is captured again when they change."""
import hashlib
import os
import re

ROOT = os.path.join(os.path.dirname(__file__), "..")
SOURCES = ("rotary.cu", "paged.cuh", "paged_rows.cu", "paged_tiles.cu", "paged_join.cu")


def digest():
    h = hashlib.sha256()
    for name in SOURCES:
        text = open(os.path.join(ROOT, "transformer_linear_layer_gb300", "csrc", name)).read()
        assert "/*" not in text  # line comments only
        h.update("".join(re.sub(r"//[^\n]*", "", text).split()).encode())
    return h.hexdigest()[:16]


def test_the_profile_is_of_these_kernels():
    text = open(os.path.join(ROOT, "profiles", "serving_operators.md")).read()
    assert re.search(r"kernel_code_sha256_16: (\w+)", text)[1] == digest()
