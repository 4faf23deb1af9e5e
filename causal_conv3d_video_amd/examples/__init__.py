"""Examples of the library used as a program would."""
