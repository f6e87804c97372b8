"""The PyTorch binding of the stored score rows is compiled again for another PyTorch or Python."""
import os

from lazy_score_matrix_gb300 import build as tpbuild


def test_binding_is_rebuilt_for_another_pytorch(monkeypatch, tmp_path):
    tpbuild.build()
    assert not tpbuild._binding_due()
    key = os.path.join(tpbuild.OBJ_DIR, "tp_logits_torch.key")
    made_for = open(key).read()
    monkeypatch.setattr(tpbuild, "_binding_key", lambda: made_for.replace("__version__", "__version__ = '0.0'  #"))
    assert tpbuild._binding_due()
    monkeypatch.undo()
    monkeypatch.setattr(tpbuild, "OBJ_DIR", str(tmp_path))  # an object of which nothing says what it was made for
    (tmp_path / "tp_logits_torch.o").write_text("")
    assert tpbuild._binding_due()
