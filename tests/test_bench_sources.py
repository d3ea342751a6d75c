"""The DRAM record of the benchmark holds for the sources of an encode: their
hash changes with any code that an encode runs, host code and new files among
them, and not with comments or with the operators beside the encode."""
import os
import shutil

import pytest

import bench

CSRC = os.path.join("exact_bpe_tokenization_utf_gb300", "csrc")
BESIDE = {"tok_paged.cu", "tok_logits.cu", "tok_grammar.cu", "tok_scan.cuh"}
FILES = sorted(f for f in os.listdir(os.path.join(bench.ROOT, CSRC)) if f.endswith((".cu", ".cuh", ".inc")))


@pytest.fixture
def tree(tmp_path, monkeypatch):
    shutil.copytree(os.path.join(bench.ROOT, CSRC), tmp_path / CSRC)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    return tmp_path / CSRC


def _append(path, text):
    with open(path, "a", encoding="utf-8") as f:
        f.write(text)


@pytest.mark.parametrize("name", FILES)
def test_code_counts_and_comments_do_not(tree, name):
    before = bench._sources_hash()
    _append(tree / name, "\n// a comment\n/* another\n */\n")
    assert bench._sources_hash() == before
    _append(tree / name, "\nint added;\n")
    assert (bench._sources_hash() == before) == (name in BESIDE)


def test_a_new_file_counts(tree):
    before = bench._sources_hash()
    (tree / "tok_new.cuh").write_text("int added;\n")
    assert bench._sources_hash() != before


def test_the_operators_beside_are_not_part_of_an_encode():
    # none of the sources of an encode includes them
    for f in FILES:
        if f not in BESIDE:
            with open(os.path.join(bench.ROOT, CSRC, f), encoding="utf-8") as fh:
                text = fh.read()
            assert not any('"%s"' % b in text for b in BESIDE), f
